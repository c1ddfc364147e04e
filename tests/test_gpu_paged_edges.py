"""Calls at the edges of what the paged-cache operators allow: graphs that begin with them or join
several streams, calls at the same time, rows that hold no numbers beside rows that do, positions and
pools past 2^30 and 2^32, outputs past 2^31 elements. Tolerances as in the other paged-cache tests."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

G = pytest.importorskip("global_interleaved_layers_b200")
from gpu_util import TOL_LSE, assert_close  # noqa: E402
from paged_util import Cache, quantise64, run_attend, turn64  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    G.gemma_attn_check()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Step:
    """An attend call with everything that it needs."""

    def __init__(self, kind, hq, hkv, d, window, dtype, nq, ctx, seed):
        self.par = G.params(kind, hq, hkv, d, window=window, rope_p=1.0 if kind == G.LOCAL else 0.25)
        self.cache = Cache(G, kind, hkv, d, 32, dtype, [n + c for n, c in zip(nq, ctx)], seed=seed)
        self.nq, self.B, self.T = nq, len(nq), sum(nq)
        self.cu, self.lens = ints([sum(nq[:i]) for i in range(len(nq) + 1)]), ints(list(ctx))
        self.max = (max(nq), max(ctx))
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q = torch.randn(self.T, hq, d, generator=gen, device="cuda").to(torch.bfloat16)
        self.src = self.q.clone()
        self.out = torch.zeros_like(self.q)
        self.need = G.gemma_attn_paged_workspace_size(self.par, self.cache.handle, self.B, self.T, *self.max)
        self.ws = torch.full((max(self.need, 256),), 255, dtype=torch.uint8, device="cuda")

    def __call__(self):
        G.gemma_attn_paged_attend(self.par, self.cache.handle, self.q, self.cu, self.lens, self.out, None, self.B, self.T,
                                  *self.max, self.ws, self.need)


def steps():
    return [Step(G.GLOBAL, 8, 1, 512, 0, "bf16", (1, 1, 1), (2000, 300, 5), 1),
            Step(G.LOCAL, 8, 4, 256, 100, "e4m3", (90, 1, 300), (40, 700, 0), 2),
            Step(G.GLOBAL, 8, 1, 512, 0, "e4m3", (200, 1, 5), (999, 2000, 64), 3),
            Step(G.GLOBAL, 4, 1, 64, 0, "bf16", (3, 1, 40), (1999, 64, 0), 4)]


def test_graphs_that_begin_with_a_call_follow_a_copy_or_join_streams():
    for s in steps():
        s()
        torch.cuda.synchronize()
        want = s.out.clone()
        side = torch.cuda.Stream()
        done = torch.cuda.Event()

        def first():
            s()

        def after_a_copy():
            s.q.copy_(s.src)
            s()

        def after_a_fill():
            s.out.zero_()
            s()
            s()

        def joined():
            here = torch.cuda.current_stream()
            side.wait_stream(here)
            with torch.cuda.stream(side):
                s.q.copy_(s.src)
                s.q.mul_(1.0)
                done.record(side)
            s.out.zero_()
            here.wait_event(done)
            s()
            s.lens.add_(0)

        for body in (first, after_a_copy, after_a_fill, joined):
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                body()
            for _ in range(3):
                if body is not first:
                    s.out.fill_(7)
                if body in (after_a_copy, joined):
                    s.q.fill_(3)
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(s.out, want), body.__name__
            s.q.copy_(s.src)
    G.gemma_attn_check()


def test_calls_at_the_same_time_on_four_streams():
    every = steps()
    for s in every:
        s()
    torch.cuda.synchronize()
    want = [s.out.clone() for s in every]
    streams = [torch.cuda.Stream() for _ in every]
    for s in every:
        s.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st in zip(every, streams):
            with torch.cuda.stream(st):
                s()
    torch.cuda.synchronize()
    for s, w in zip(every, want):
        assert torch.equal(s.out, w)
    G.gemma_attn_check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,hq,hkv,d", [(G.GLOBAL, 8, 1, 512), (G.LOCAL, 8, 2, 128), (G.LOCAL, 4, 1, 64), (G.GLOBAL, 8, 1, 256)])
def test_query_rows_without_numbers_leave_the_others_alone(kind, hq, hkv, d, dtype):
    par = G.params(kind, hq, hkv, d, window=50 if kind == G.LOCAL else 0, rope_p=1.0 if kind == G.LOCAL else 0.25)
    for nq, ctx in (((1, 1), (70, 300)), ((5, 2), (70, 300)), ((40, 90), (70, 300))):
        cache = Cache(G, kind, hkv, d, 16, dtype, [n + c for n, c in zip(nq, ctx)], seed=4)
        q = torch.randn(sum(nq), hq, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
        want, want_lse = run_attend(G, cache, par, q, nq, ctx)
        bad = torch.zeros(sum(nq), hq, dtype=torch.bool, device="cuda")
        bad[::3, 1::3] = True
        x = q.clone()
        x[bad] = torch.where(torch.arange(d, device="cuda") % 7 == 3, math.nan, x[bad])
        bad[0, 0] = True
        x[0, 0, 5] = math.inf
        got, lse = run_attend(G, cache, par, x, nq, ctx)
        G.gemma_attn_check()
        assert torch.equal(got[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])
        assert bool(torch.isnan(got[bad]).all()) and bool(torch.isnan(lse[bad]).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,nq", [(256, 1), (256, 5), (256, 100), (64, 2)])
def test_far_positions_in_a_large_pool(d, nq, dtype):
    """Positions past 2^30 and pages whose bytes lie past 2^32: a sliding-window layer needs only the
    table entries and pages of its window. The angle of a position below 2^31 is formed in 64 bits,
    its rounding to fp32 half turns is the same as nearer by."""
    page, window, ctx = 256, 300, (1 << 30) + 77
    size = 1 if dtype == "e4m3" else 2
    num = (1 << 32) // (page * d * size) + 1000
    n0 = ctx - window + 1
    par = G.params(G.LOCAL, 2, 1, d, window=window, rope_p=1.0)
    par.out_dtype = G.OUT_F32
    table = torch.full((1, (ctx + nq) // page + 1), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(n0 // page, (ctx + nq - 1) // page + 1, device="cuda")
    table[0, used] = (num - 1 - 3 * torch.arange(len(used), device="cuda")).to(torch.int32)
    dt = torch.float8_e4m3fn if dtype == "e4m3" else torch.bfloat16
    pools = [torch.empty(num, 1, page, d, dtype=dt, device="cuda") for _ in range(2)]
    scales = [torch.empty(num, 1, page, device="cuda") if dtype == "e4m3" else None for _ in range(2)]
    cache = G.paged_cache(pools[0], pools[1], table, k_scales=scales[0], v_scales=scales[1])
    gen = torch.Generator().manual_seed(3)
    total = ctx + nq - n0
    k, v = (torch.randn(total, 1, d, generator=gen).to(torch.bfloat16) for _ in range(2))
    G.gemma_attn_paged_append(par, cache, k.cuda(), v.cuda(), ints([0, total]), ints([n0]), 1, total)
    back = [torch.empty(total, 1, d, device="cuda") for _ in range(2)]
    G.gemma_attn_paged_gather(par, cache, ints([n0]), ints([0, total]), back[0], back[1], 1, total)
    G.gemma_attn_check()
    pos = torch.arange(n0, ctx + nq, dtype=torch.int64)
    kk, vv = turn64(k.double(), pos, d // 2, par.rope_base), v.double()
    if dtype == "e4m3":
        assert torch.equal(back[1].cpu().double(), quantise64(vv)[0])
        step = 2.0 ** -3
    else:
        assert torch.equal(back[1].cpu().double(), vv)
        step = 2.0 ** -7
    got = back[0].cpu().double()
    assert bool(((got - kk).abs() <= kk.abs() * step + kk.abs().amax(-1, keepdim=True) * 2.0 ** (-20 if size == 2 else -14)).all())
    q = torch.randn(nq, 2, d, generator=gen).to(torch.bfloat16)
    out, lse = torch.empty(nq, 2, d, device="cuda"), torch.empty(nq, 2, device="cuda")
    need = G.gemma_attn_paged_workspace_size(par, cache, 1, nq, nq, ctx)
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
    G.gemma_attn_paged_attend(par, cache, q.cuda(), ints([0, nq]), ints([ctx]), out, lse, 1, nq, nq, ctx, ws, need)
    G.gemma_attn_check()
    pq = torch.arange(ctx, ctx + nq, dtype=torch.int64)
    s = torch.einsum("nhd,kd->nhk", turn64(q.double(), pq, d // 2, par.rope_base), got[:, 0]) * par.softmax_scale
    hide = (pos[None] > pq[:, None]) | (pos[None] <= pq[:, None] - window)
    s = s.masked_fill(hide[:, None], -math.inf)
    ref = torch.einsum("nhk,kd->nhd", torch.softmax(s, -1), back[1].cpu().double()[:, 0])
    assert_close(out.cpu().numpy(), ref.numpy(), "far away")
    assert float((lse.cpu().double() - torch.logsumexp(s, -1)).abs().max()) <= TOL_LSE


def test_an_output_past_2_to_31_elements():
    n, hq, d, page, window = 131072 + 300, 32, 512, 256, 33
    par = G.params(G.LOCAL, hq, 1, d, window=window, rope_p=0.25)
    blocks = -(-n // page)
    gen = torch.Generator(device="cuda").manual_seed(1)
    pools = [torch.randn(blocks, 1, page, d, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").view(1, -1)
    cache = G.paged_cache(pools[0], pools[1], table)
    q = torch.randn(n, hq, d, generator=gen, device="cuda", dtype=torch.bfloat16)
    out = torch.empty_like(q)
    assert out.numel() > 1 << 31
    need = G.gemma_attn_paged_workspace_size(par, cache, 1, n, n, 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    G.gemma_attn_paged_attend(par, cache, q, ints([0, n]), ints([0]), out, None, 1, n, n, 0, ws, need)
    G.gemma_attn_check()
    for a in (0, 65000, n - 40):
        b, lo = a + 40, max(0, a - window + 1)
        k, v = (x.view(-1, d)[lo:b].double() for x in pools)
        s = torch.einsum("nhd,kd->nhk", turn64(q[a:b].double(), torch.arange(a, b, device="cuda"), d // 8, par.rope_base), k)
        i, j = torch.arange(a, b, device="cuda")[:, None, None], torch.arange(lo, b, device="cuda")
        s = (s * par.softmax_scale).masked_fill((j > i) | (j <= i - window), -math.inf)
        ref = torch.einsum("nhk,kd->nhd", torch.softmax(s, -1), v)
        # bf16 outputs: half a step of values that reach 4, beside the usual bound
        diff = (out[a:b].double() - ref).abs()
        assert float(diff.max()) <= 1e-2 + 2.0 ** -8 * 4 and float(diff.norm() / ref.norm()) <= 5e-3
