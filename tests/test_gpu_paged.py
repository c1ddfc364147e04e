"""Paged-cache operators on the GPU against 64-bit implementations: append, read back, attention.

Tolerances. Read-back rows: equal where nothing is rotated. Rotated keys: the fp32 rotation is
off by at most 2^-20 of the row's largest element (the angle by pi 2^-24 from its rounding to fp32
half turns, cosine and sine by 2^-23, product and difference by 3 x 2^-24: under 2^-21 of the
pair's length, which is at most sqrt(2) of the largest element), then one rounding; so each
element is within half a step of its type (bf16: 2^-8, e4m3: 2^-4 of its value) plus the
neighbour that such a nudge can tip it to: one whole step and 2^-20 of the largest element,
the nudge itself where cancellation leaves a value that small. All but a small share are equal.
Attention in fp32 output: the acceptance bounds of the prefill and decode kernels (max-abs 1e-2,
relative RMS 5e-3: rotated queries and keys and the weights are rounded to bf16, 2^-8 of a value
each at most, on unit-normal inputs); the log-sum-exp 1e-2 as theirs.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

G = pytest.importorskip("global_interleaved_layers_b200")
from gpu_util import TOL_LSE, assert_close  # noqa: E402
from paged_util import Cache, attend64, quantise64, run_attend, turn64  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    G.gemma_attn_check()


def params(kind, hq, hkv, d, window=0, p=None, base=None):
    return G.params(kind, hq, hkv, d, window=window, rope_p=(1.0 if kind == G.LOCAL else 0.25) if p is None else p,
                    rope_base=(1e4 if kind == G.LOCAL else 1e6) if base is None else base)


def cu_of(ns):
    return torch.tensor([0] + list(np.cumsum(ns)), dtype=torch.int32, device="cuda")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------- append and read back

@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,hkv,d,page,p", [
    (G.LOCAL, 3, 64, 16, 1.0), (G.LOCAL, 2, 128, 32, 0.5), (G.LOCAL, 16, 256, 64, 1.0), (G.LOCAL, 1, 512, 256, 1.0),
    (G.LOCAL, 2, 256, 16, 0.0), (G.LOCAL, 2, 256, 16, 0.03), (G.GLOBAL, 1, 512, 128, 0.25), (G.GLOBAL, 5, 64, 16, 0.25),
])
@pytest.mark.parametrize("nq,ctx", [((1,), (0,)), ((3, 0, 40, 1, 17), (0, 5, 33, 16, 4000))])
def test_append_then_gather(dtype, kind, hkv, d, page, p, nq, ctx):
    par = params(kind, hkv, hkv, d, window=64, p=p)
    cache = Cache(G, kind, hkv, d, page, dtype, [n + c for n, c in zip(nq, ctx)], seed=1, keep=[c // page * page for c in ctx])
    before = {t: x.clone() for t, x in cache.pages.items()}
    T = sum(nq)
    new = {t: torch.randn(T + 2, hkv, d, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda()
           for i, t in enumerate(cache.pages)}
    # two rows past the last sequence: not stored
    G.gemma_attn_paged_append(par, cache.handle, new["k"], new.get("v"), cu_of(nq), ints(ctx), len(nq), T + 2)
    assert G.gemma_attn_last_launch_count() == 1
    back = {t: torch.full((T + 2, hkv, d), 7.0, device="cuda") for t in cache.pages}
    pf = G.GemmaAttnParams.from_buffer_copy(par)
    pf.out_dtype = G.OUT_F32
    G.gemma_attn_paged_gather(pf, cache.handle, ints(ctx), cu_of(nq), back["k"], back.get("v"), len(nq), T + 2)
    b16 = {t: torch.full((T + 2, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for t in cache.pages}
    G.gemma_attn_paged_gather(par, cache.handle, ints(ctx), cu_of(nq), b16["k"], b16.get("v"), len(nq), T + 2)
    G.gemma_attn_check()
    pos = torch.cat([torch.arange(c, c + n, device="cuda") for n, c in zip(nq, ctx)])
    r = int(p * d / 2) if kind == G.LOCAL else 0
    for t in cache.pages:
        want = new[t][:T].double()
        turned = t == "k" and r > 0
        if turned:
            want = turn64(want, pos, r, 1e4)
        got = back[t][:T].double()
        assert torch.equal(back[t], torch.cat([back[t][:T], torch.full_like(back[t][T:], 7.0)]))  # padding rows untouched
        assert torch.equal(b16[t].float(), back[t])  # exact in bf16
        if dtype == "e4m3":
            want = quantise64(want)[0]
        else:
            want = want.float().to(torch.bfloat16).double()
        if not turned:
            assert torch.equal(got, want)
        else:
            one = 2.0 ** (-3 if dtype == "e4m3" else -7)  # a whole step
            amax = want.abs().amax(-1, keepdim=True)
            tiny = amax / 448 * 2.0 ** -6 if dtype == "e4m3" else torch.zeros_like(amax)  # e4m3's fixed step at the bottom
            most = torch.maximum(torch.maximum(got.abs(), want.abs()) * one, tiny) + amax * 2.0 ** -20
            assert bool(((got - want).abs() <= most).all())
            # a nudge of 2^-22 tips one rounding in 2^13 at bf16's steps
            assert int((got != want).sum()) <= 8 + got.numel() // 1000
    # every other row of the pool is as it was
    for t, was in before.items():
        now, old = cache.pages[t].view(torch.uint8 if dtype == "e4m3" else torch.int16), was.view(torch.uint8 if dtype == "e4m3" else torch.int16)
        touched = torch.zeros(cache.num_pages, page, dtype=torch.bool, device="cuda")
        for b, (n, c) in enumerate(zip(nq, ctx)):
            for q in range(c, c + n):
                touched[int(cache.table[b, q // page]), q % page] = True
        same = (now == old).all(-1)  # [pages, heads, slots]
        assert bool((same | touched[:, None]).all())


def test_quantised_rows_at_their_limits():
    """Scale borders, zero rows, subnormals, the largest bf16 values, infinities and NaN."""
    d, page = 64, 16
    par = params(G.GLOBAL, 1, 1, d)
    x = torch.randn(12, 1, d, generator=torch.Generator().manual_seed(3)).clamp(-3, 3)
    x[0] = 0
    x[1, 0, 5] = 448.0       # scale 1
    x[2, 0, 5] = 450.0       # scale 2
    x[3] *= 2.0 ** -130      # below the smallest scale's range: e4m3 steps of 2^-135
    x[4] *= 2.0 ** 125
    x[5, 0, 7] = math.inf
    x[6, 0, 60] = math.nan
    x[7, 0, 33] = -math.inf
    x[8] = 3.3895313892515355e38  # the largest bf16
    x[9, 0, 0] = -448.0 * 2.0 ** -9
    x[10] *= 1e-3
    x = x.to(torch.bfloat16)
    cache = Cache(G, G.GLOBAL, 1, d, page, "e4m3", [12], seed=1)
    G.gemma_attn_paged_append(par, cache.handle, x.cuda(), None, cu_of([12]), ints([0]), 1, 12)
    pf = G.GemmaAttnParams.from_buffer_copy(par)
    pf.out_dtype = G.OUT_F32
    back = torch.empty(12, 1, d, device="cuda")
    G.gemma_attn_paged_gather(pf, cache.handle, ints([0]), cu_of([12]), back, None, 1, 12)
    G.gemma_attn_check()
    finite = [i for i in range(12) if i not in (5, 6, 7)]
    want = quantise64(x.double())[0]
    wrong = (back.cpu().double() != want).flatten(1).sum(1)
    assert wrong[finite].tolist() == [0] * 9
    assert torch.isnan(back[[5, 6, 7]]).all()
    scale = cache.scales["k"][int(cache.table[0, 0]), 0, :12].cpu()
    assert scale[0] == 1 and scale[1] == 1 and scale[2] == 2 and torch.isnan(scale[[5, 6, 7]]).all()
    assert scale[3] == 2.0 ** -126 and scale[8] == 2.0 ** 120
    assert not cache.pages["k"][int(cache.table[0, 0]), 0, [5, 6, 7]].view(torch.uint8).any()


def test_append_and_gather_record_bad_positions_and_pages():
    d, page = 64, 16
    par = params(G.GLOBAL, 1, 1, d)
    cache = Cache(G, G.GLOBAL, 1, d, page, "bf16", [40], seed=1)
    x = torch.randn(4, 1, d, device="cuda").to(torch.bfloat16)
    was = cache.pages["k"].clone()
    for ctx, code in ((cache.max_blocks * page - 3, G.ERR_PAGE), (cache.max_blocks * page, G.ERR_SEQLEN), (-5, G.ERR_SEQLEN)):
        G.gemma_attn_paged_append(par, cache.handle, x, None, cu_of([3]), ints([ctx]), 1, 4)
        with pytest.raises(G.GemmaAttnError) as e:
            G.gemma_attn_check()
        assert e.value.status == code
        assert torch.equal(cache.pages["k"].view(torch.int16), was.view(torch.int16))
        out = torch.full((3, 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
        G.gemma_attn_paged_gather(par, cache.handle, ints([ctx]), cu_of([3]), out, None, 1, 3)
        with pytest.raises(G.GemmaAttnError) as e:
            G.gemma_attn_check()
        assert e.value.status == code and not out.any()


# ---------------------------------------------------------------------------- attention

def check_attend(kind, hq, hkv, d, page, dtype, nq, ctx, window=0, p=None, pad_rows=0, max_q=None, max_len=None, seed=0,
                 scale=1.0):
    par = params(kind, hq, hkv, d, window=window, p=p)
    # pages wholly before the oldest query's window are dropped
    keep = [max(0, c - window + 1) if window else 0 for c in ctx]
    cache = Cache(G, kind, hkv, d, page, dtype, [n + c if n else c for n, c in zip(nq, ctx)], seed=seed, keep=keep, scale=scale)
    q = torch.randn(sum(nq) + pad_rows, hq, d, generator=torch.Generator().manual_seed(seed + 99)).to(torch.bfloat16).cuda()
    out, lse = run_attend(G, cache, par, q, nq, ctx, pad_rows=pad_rows, max_q=max_q, max_len=max_len)
    out16, _ = run_attend(G, cache, par, q, nq, ctx, out_f32=False, pad_rows=pad_rows, lse=False, max_q=max_q, max_len=max_len)
    G.gemma_attn_check()
    r = int(par.rope_p * d / 2)
    at = 0
    for b, (n, c) in enumerate(zip(nq, ctx)):
        if n == 0:
            continue
        k = cache.rows["k"][b]
        ref, ref_lse = attend64(q[at:at + n].double(), k, k if kind == G.GLOBAL else cache.rows["v"][b], c, window, r,
                                par.rope_base, par.softmax_scale, kind == G.GLOBAL)
        got = out[at:at + n]
        assert_close(got.cpu().numpy() / scale, ref.cpu().numpy() / scale, f"sequence {b}: {n} tokens after {c}")
        assert float((lse[at:at + n].double() - ref_lse).abs().max()) <= TOL_LSE * max(1.0, scale)
        at += n
    assert bool((out[at:] == 7).all()) and bool((out16[at:] == 7).all())
    assert torch.equal(out16[:at], out[:at].to(torch.bfloat16))
    return out


LAYERS = [
    (G.LOCAL, 8, 4, 256, 32, 100), (G.LOCAL, 6, 2, 64, 16, 37), (G.LOCAL, 12, 1, 128, 256, 1), (G.LOCAL, 16, 16, 512, 64, 300),
    (G.GLOBAL, 8, 1, 512, 64, 0), (G.GLOBAL, 16, 2, 256, 16, 0), (G.GLOBAL, 20, 4, 128, 128, 0), (G.GLOBAL, 8, 1, 64, 32, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,hq,hkv,d,page,window", LAYERS)
def test_decode_one_token(kind, hq, hkv, d, page, window, dtype):
    check_attend(kind, hq, hkv, d, page, dtype, (1, 1, 1, 1, 1, 1, 1), (0, 1, 15, 16, 17, 301, 1000), window)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,hq,hkv,d,page,window", LAYERS)
def test_ragged_chunks_with_empty_sequences_and_padding(kind, hq, hkv, d, page, window, dtype):
    check_attend(kind, hq, hkv, d, page, dtype, (0, 3, 1, 0, 130, 17, 0), (9, 0, 500, 0, 77, 128, 3), window, pad_rows=5,
                 max_q=200, max_len=2000)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,hq,hkv,d,page,window,n,c", [
    (G.GLOBAL, 8, 1, 512, 64, 0, 600, 700), (G.LOCAL, 4, 2, 256, 16, 200, 700, 450), (G.GLOBAL, 3, 1, 128, 16, 0, 511, 1),
    (G.LOCAL, 1, 1, 64, 128, 513, 1300, 0),
])
def test_long_chunk(kind, hq, hkv, d, page, window, n, c, dtype):
    check_attend(kind, hq, hkv, d, page, dtype, (n,), (c,), window)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq", [(1, 1), (5, 4), (40, 1)])
def test_long_history_is_split(nq, dtype):
    check_attend(G.GLOBAL, 8, 1, 512, 64, dtype, nq, (20011, 333))


@pytest.mark.parametrize("p", [0.0, 0.03, 0.6, 1.0])
@pytest.mark.parametrize("d", [64, 512])
def test_rotated_fraction(p, d):
    for dtype in ("bf16", "e4m3"):
        check_attend(G.GLOBAL, 4, 1, d, 16, dtype, (1, 33), (70, 40), p=p)


@pytest.mark.parametrize("scale", [2.0 ** -20, 2.0 ** 18])
def test_rows_of_any_size(scale):
    """Values far from 1: separate keys are unit rows, values and K=V rows are not. For large K=V
    rows the softmax is a maximum; rows stay within it in relative terms."""
    par = params(G.LOCAL, 2, 1, 128, window=64)
    for dtype in ("bf16", "e4m3"):
        cache = Cache(G, G.LOCAL, 1, 128, 16, dtype, [100], seed=5)
        if dtype == "bf16":
            cache.pages["v"].mul_(scale)
        else:
            cache.scales["v"].mul_(scale)
        q = torch.randn(1, 2, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
        out, _ = run_attend(G, cache, par, q, (1,), (99,))
        ref, _ = attend64(q.double(), cache.rows["k"][0], cache.rows["v"][0], 99, 64, 64, 1e4, par.softmax_scale, False)
        G.gemma_attn_check()
        assert_close(out.cpu().numpy() / scale, ref.cpu().numpy(), dtype)


@pytest.mark.parametrize("nq", [1, 60])
def test_value_scales_that_differ_between_keys(nq):
    """e4m3 values whose scales span 2^60: the keys with the large weights have the tiny values,
    one far key the large ones; and a key with tiny values only must not disturb the sum.

    Outputs then reach many times their mean square, so the bound is per element. With no
    rotation the scores are exact products summed in fp32 (about 2^-20 absolute: 2^-16 of a
    weight with the exponential's own error, generously). Each weight is then rounded to 16 bits,
    by half a step, 2^-8 of itself in bf16 (2^-11 in fp16), the sum is not: an output is off by
    at most (2^-8 + 2^-16) sum p|v|. fp16 weights under 2^-14 of the largest keep 2^-25 of it, against codes of
    at most 448 beside one of at least 224: 2^-20 of the row's largest sum covers 200 such keys."""
    par = params(G.LOCAL, 2, 1, 64, window=4096, p=0.0)
    cache = Cache(G, G.LOCAL, 1, 64, 16, "e4m3", [200], seed=5)
    f = torch.ones(200, dtype=torch.float64)
    f[::3], f[1::5], f[7] = 2.0 ** -30, 2.0 ** 30, 2.0 ** -90
    for i in range(200):
        cache.scales["v"][int(cache.table[0, i // 16]), :, i % 16] *= float(f[i])
    q = 3 * torch.randn(nq, 2, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    out, lse = run_attend(G, cache, par, q, (nq,), (200 - nq,))
    ref, ref_lse = attend64(q.double(), cache.rows["k"][0], cache.rows["v"][0] * f.cuda()[:, None, None], 200 - nq, 4096, 0, 1e4,
                            par.softmax_scale, False)
    G.gemma_attn_check()
    size, _ = attend64(q.double(), cache.rows["k"][0], (cache.rows["v"][0] * f.cuda()[:, None, None]).abs(), 200 - nq, 4096, 0, 1e4,
                       par.softmax_scale, False)
    most = (2.0 ** -8 + 2.0 ** -16) * size + 2.0 ** -20 * size.amax(-1, keepdim=True) * 2
    assert bool(((out.double() - ref).abs() <= most).all())
    assert float((lse.double() - ref_lse).abs().max()) <= TOL_LSE


def test_quantised_attention_is_attention_over_the_rows_read_back():
    for kind, window in ((G.GLOBAL, 0), (G.LOCAL, 150)):
        nq, ctx = (1, 40, 3), (333, 100, 0)
        par = params(kind, 8, 2, 256, window=window)
        c8 = Cache(G, kind, 2, 256, 32, "e4m3", [n + c for n, c in zip(nq, ctx)], seed=4)
        c16 = Cache(G, kind, 2, 256, 32, "bf16", [n + c for n, c in zip(nq, ctx)], seed=4)
        tot = [n + c for n, c in zip(nq, ctx)]
        back = [torch.empty(sum(tot), 2, 256, dtype=torch.bfloat16, device="cuda") for _ in c8.pages] + [None]
        G.gemma_attn_paged_gather(par, c8.handle, ints([0, 0, 0]), cu_of(tot), back[0], back[1], 3, sum(tot))
        par0 = params(kind, 8, 2, 256, window=window, p=0.0)  # rows are stored as read: no second rotation
        G.gemma_attn_paged_append(par0, c16.handle, back[0], back[1], cu_of(tot), ints([0, 0, 0]), 3, sum(tot))
        q = torch.randn(sum(nq), 8, 256, device="cuda").to(torch.bfloat16)
        a, la = run_attend(G, c8, par, q, nq, ctx)
        b, lb = run_attend(G, c16, par, q, nq, ctx)
        G.gemma_attn_check()
        assert_close(a.cpu().numpy(), b.cpu().double().numpy(), "e4m3 against its read-back")
        assert float((la - lb).abs().max()) <= TOL_LSE


def test_bad_table_entries_and_lengths_are_recorded():
    par = params(G.GLOBAL, 8, 1, 64)
    cache = Cache(G, G.GLOBAL, 1, 64, 16, "bf16", [100, 64], seed=2)
    q = torch.randn(2, 8, 64, device="cuda").to(torch.bfloat16)
    good, _ = run_attend(G, cache, par, q, (1, 1), (99, 63))
    G.gemma_attn_check()
    cache.table[0, 2] = cache.num_pages  # positions 32..47 of the first sequence
    out, _ = run_attend(G, cache, par, q, (1, 1), (99, 63))
    with pytest.raises(G.GemmaAttnError) as e:
        G.gemma_attn_check()
    assert e.value.status == G.ERR_PAGE
    assert torch.equal(out[1], good[1])
    rows = torch.cat([cache.rows["k"][0][:32], cache.rows["k"][0][48:]])
    kk = torch.cat([turn64(cache.rows["k"][0], torch.arange(100, device="cuda"), 8, 1e6)[s] for s in (slice(0, 32), slice(48, 100))])
    qq = turn64(q[:1].double(), torch.tensor([99], device="cuda"), 8, 1e6)
    s = torch.softmax(torch.einsum("nhd,kd->nhk", qq, kk[:, 0]) * par.softmax_scale, -1)
    assert_close(out[:1].cpu().numpy(), torch.einsum("nhk,kd->nhd", s, rows[:, 0]).cpu().numpy(), "without the bad page")
    cache.table[0, 2] = -1
    run_attend(G, cache, par, q, (1, 1), (99, 63))
    with pytest.raises(G.GemmaAttnError) as e:
        G.gemma_attn_check()
    assert e.value.status == G.ERR_PAGE
    # lengths past the stated bounds, past the table, negative: recorded, rows not written
    for nq, ctx, mq, ml in (((1, 1), (99, 63), 1, 98), ((2,), (60,), 1, 200), ((1, 1), (16 * cache.max_blocks, 63), 1, 10000),
                            ((1, 1), (-1, 63), 1, 200)):
        out, _ = run_attend(G, cache, par, q, nq, ctx, max_q=mq, max_len=ml)
        with pytest.raises(G.GemmaAttnError) as e:
            G.gemma_attn_check()
        assert e.value.status == G.ERR_SEQLEN
        assert bool((out[0] == 7).all())
    # a prefix that runs past the rows given
    out = torch.full((2, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    nb = G.gemma_attn_paged_workspace_size(par, cache.handle, 2, 2, 64, 64)
    ws = torch.empty(max(nb, 256), dtype=torch.uint8, device="cuda")
    G.gemma_attn_paged_attend(par, cache.handle, q, ints([0, 1, 40]), ints([5, 5]), out, None, 2, 2, 64, 64, ws, nb)
    with pytest.raises(G.GemmaAttnError) as e:
        G.gemma_attn_check()
    assert e.value.status == G.ERR_SEQLEN and bool((out[1] == 7).all())


def test_captured_and_replayed_and_on_two_streams():
    """A serving step (append, attention) captured once: replays follow new rows and lengths, and two
    graphs with a workspace each may run at the same time."""
    cases = []
    for i, (kind, window, nq) in enumerate(((G.GLOBAL, 0, (1, 1, 1)), (G.LOCAL, 100, (9, 30, 2)))):
        par = params(kind, 8, 1, 512 if kind == G.GLOBAL else 256, window=window)
        cache = Cache(G, kind, 1, par.head_dim, 32, ("bf16", "e4m3")[i], [9000, 777, 4000], seed=i)
        T = sum(nq)
        s = {"par": par, "cache": cache, "nq": nq, "lens": ints([100, 50, 7]), "cu": cu_of(nq),
             "q": torch.randn(T, 8, par.head_dim, device="cuda").to(torch.bfloat16), "out": torch.empty(T, 8, par.head_dim, dtype=torch.bfloat16, device="cuda"),
             "new": [torch.randn(T, 1, par.head_dim, device="cuda").to(torch.bfloat16) for _ in cache.pages] + [None]}
        s["nb"] = G.gemma_attn_paged_workspace_size(par, cache.handle, 3, T, max(nq), 9000)
        s["ws"] = torch.empty(max(s["nb"], 256), dtype=torch.uint8, device="cuda")
        cases.append(s)

    def step(s):
        G.gemma_attn_paged_append(s["par"], s["cache"].handle, s["new"][0], s["new"][1], s["cu"], s["lens"], 3, sum(s["nq"]))
        G.gemma_attn_paged_attend(s["par"], s["cache"].handle, s["q"], s["cu"], s["lens"], s["out"], None, 3, sum(s["nq"]),
                                  max(s["nq"]), 9000, s["ws"], s["nb"])

    graphs = []
    for s in cases:
        step(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens in ([100, 50, 7], [8000, 0, 3900], [31, 32, 33]):
        want = []
        for s in cases:
            s["lens"].copy_(ints(lens))
            s["q"].normal_()
            step(s)
            torch.cuda.synchronize()
            want.append(s["out"].clone())
            s["out"].fill_(7)
        torch.cuda.synchronize()
        for _ in range(3):
            for st, g in zip(streams, graphs):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for s, w in zip(cases, want):
            assert torch.equal(s["out"], w)
    G.gemma_attn_check()


def test_a_stream_of_its_own():
    par = params(G.GLOBAL, 8, 1, 128)
    cache = Cache(G, G.GLOBAL, 1, 128, 16, "bf16", [500], seed=2)
    q = torch.randn(1, 8, 128, device="cuda").to(torch.bfloat16)
    want, _ = run_attend(G, cache, par, q, (1,), (499,))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got, _ = run_attend(G, cache, par, q, (1,), (499,), stream=st)
    st.synchronize()
    assert torch.equal(got, want)
