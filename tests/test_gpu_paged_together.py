"""The paged-cache operators and the draft verification as a serving loop uses them, and calls
at the edges of what they allow. Attention tolerances are those of the paged-cache tests: max-abs
1e-2 and relative RMS 5e-3 on unit-normal inputs, log-sum-exp 1e-2."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

G = pytest.importorskip("global_interleaved_layers_b200")
from gpu_util import TOL_LSE, assert_close  # noqa: E402
from paged_util import attend64, quantise64, turn64  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    G.gemma_attn_check()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cu_of(ns):
    return ints([0] + [int(x) for x in np.cumsum(ns)])


class Layer:
    """A layer with its pages, and the rows that it was given, by sequence."""

    def __init__(self, kind, hq, hkv, d, window, dtype, page, batch, blocks, seed):
        self.kind, self.hq, self.hkv, self.d, self.window, self.dtype = kind, hq, hkv, d, window, dtype
        self.p = G.params(kind, hq, hkv, d, window=window, rope_p=1.0 if kind == G.LOCAL else 0.25,
                          rope_base=1e4 if kind == G.LOCAL else 1e6)
        self.p.out_dtype = G.OUT_F32
        self.gen = torch.Generator().manual_seed(seed)
        pages = batch * blocks
        shape = (pages, hkv, page, d)
        # what a page holds before it is written is nobody's business
        if dtype == "e4m3":
            make = lambda: torch.full(shape, float("nan")).to(torch.float8_e4m3fn).cuda()  # noqa: E731
            scales = [torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2)]
        else:
            make = lambda: torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
            scales = [None, None]
        local = kind == G.LOCAL
        self.table = torch.randperm(pages, generator=self.gen).to(torch.int32).view(batch, blocks).cuda()
        self.cache = G.paged_cache(make(), make() if local else None, self.table, k_scales=scales[0],
                                   v_scales=scales[1] if local else None)
        self.rows = [torch.zeros(0, hkv, d, dtype=torch.float64) for _ in range(batch)]
        self.vals = [torch.zeros(0, hkv, d, dtype=torch.float64) for _ in range(batch)]

    def held(self, x, at, rotate):
        x = x.double()
        if rotate:
            x = turn64(x, torch.arange(at, at + len(x)), int(self.p.rope_p * self.d / 2), self.p.rope_base)
            x = x.to(torch.bfloat16).double() if self.dtype == "bf16" else x
        return quantise64(x)[0] if self.dtype == "e4m3" else x

    def step(self, nq, lens, max_q, max_len, pad):
        """Appends nq[b] new tokens after lens[b] and attends from them; checks every sequence."""
        T = sum(nq) + pad
        new = [torch.randn(T, self.hkv, self.d, generator=self.gen).to(torch.bfloat16) for _ in range(2)]
        q = torch.randn(T, self.hq, self.d, generator=self.gen).to(torch.bfloat16)
        cu, dev_lens, local = cu_of(nq), ints(lens), self.kind == G.LOCAL
        B = len(nq)
        G.gemma_attn_paged_append(self.p, self.cache, new[0].cuda(), new[1].cuda() if local else None, cu, dev_lens, B, T)
        out = torch.full((T, self.hq, self.d), 7.0, device="cuda")
        lse = torch.full((T, self.hq), 7.0, device="cuda")
        need = G.gemma_attn_paged_workspace_size(self.p, self.cache, B, T, max_q, max_len)
        ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
        G.gemma_attn_paged_attend(self.p, self.cache, q.cuda(), cu, dev_lens, out, lse, B, T, max_q, max_len, ws, need)
        G.gemma_attn_check()
        at = 0
        for b, (n, c) in enumerate(zip(nq, lens)):
            if n == 0:
                continue
            self.rows[b] = torch.cat([self.rows[b][:c], self.held(new[0][at:at + n], c, local)])
            if local:
                self.vals[b] = torch.cat([self.vals[b][:c], self.held(new[1][at:at + n], c, False)])
            k = self.rows[b]
            ref, ref_lse = attend64(q[at:at + n].double(), k, self.vals[b] if local else k, c, self.window,
                                    int(self.p.rope_p * self.d / 2), self.p.rope_base, self.p.softmax_scale, not local)
            assert_close(out[at:at + n].cpu().numpy(), ref.numpy(), f"sequence {b}: {n} tokens after {c}")
            assert float((lse[at:at + n].cpu().double() - ref_lse).abs().max()) <= TOL_LSE
            at += n
        assert bool((out[at:] == 7).all()) and bool((lse[at:] == 7).all())


# The rotated e4m3 keys of the reference are rounded from 64 bits, the kernel's from fp32: where the
# two straddle a border they differ by an e4m3 step, 2^-3 of one element in some thousands. A
# score then moves by 2^-3 / sqrt(d) of a product of unit normals at most, far inside the bounds.
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prompts_then_drafted_tokens_are_verified_and_the_rest_overwritten(dtype):
    B, n, V = 3, 4, 301
    layers = [Layer(G.LOCAL, 4, 2, 256, 70, dtype, 16, B, 16, 1), Layer(G.GLOBAL, 8, 1, 512, 0, dtype, 64, B, 4, 2)]
    rng = np.random.default_rng(5)
    lens = [0, 0, 0]
    prompts = [90, 1, 33]
    for layer in layers:
        layer.step(prompts, lens, 128, 0, pad=7)
    lens = prompts
    for turn in range(4):
        # the last accepted token and up to four drafted ones; one sequence sits a turn out
        drafts = [int(x) for x in rng.integers(0, n + 1, B)]
        nq = [0 if b == turn else 1 + drafts[b] for b in range(B)]
        for layer in layers:
            layer.step(nq, lens, n + 1, 256, pad=turn)
        target = torch.softmax(torch.tensor(rng.standard_normal((B, n + 1, V)), dtype=torch.float32), -1).cuda()
        draft = torch.softmax(torch.log(target[:, :n]) + 0.5 * torch.randn(B, n, V, device="cuda"), -1)
        tokens = torch.multinomial(draft.view(-1, V), 1).view(B, n).to(torch.int32)
        acc, nxt = ints([0] * B), torch.zeros(B, n + 1, dtype=torch.int32, device="cuda")
        G.gemma_attn_draft_verify(target, draft, tokens, ints(drafts), torch.rand(B, n, device="cuda"),
                                  torch.empty(B, V, device="cuda").exponential_(), acc, nxt)
        G.gemma_attn_check()
        acc = acc.tolist()
        assert all(0 <= a <= d for a, d in zip(acc, drafts))
        # rejected tokens' rows stay in the pages, past the new length, and are overwritten next turn
        lens = [c if q == 0 else c + 1 + a for c, q, a in zip(lens, nq, acc)]
    starts, count = [0] * B, [min(c, 50) for c in lens]
    for layer in layers:
        out = [torch.zeros(sum(count), layer.hkv, layer.d, device="cuda") for _ in range(2)]
        G.gemma_attn_paged_gather(layer.p, layer.cache, ints(starts), cu_of(count), out[0], out[1] if layer.kind == G.LOCAL else None,
                                  B, sum(count))
        G.gemma_attn_check()
        at = 0
        for b, c in enumerate(count):
            got = out[0][at:at + c].cpu().double()
            want = layer.rows[b][:c]
            # rotated keys may land on the neighbouring number of their type
            step = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -3
            tol = want.abs() * step + want.abs().amax(-1, keepdim=True) * 2.0 ** (-20 if dtype == "bf16" else -14)
            assert bool(((got - want).abs() <= (tol if layer.kind == G.LOCAL else 0)).all())
            if layer.kind == G.LOCAL:
                assert torch.equal(out[1][at:at + c].cpu().double(), layer.vals[b][:c])
            at += c


@pytest.mark.parametrize("kind,d,window", [(G.LOCAL, 128, 9), (G.GLOBAL, 64, 0)])
def test_thousands_of_sequences_most_of_them_empty(kind, d, window):
    rng = np.random.default_rng(3)
    B = 2500
    nq = [int(x) for x in rng.choice([0, 0, 0, 1, 2], B)]
    layer = Layer(kind, 2, 1, d, window, "bf16", 16, B, 2, 4)
    layer.step(nq, [0] * B, 2, 20, pad=3)
    lens = nq
    nq = [int(x) for x in rng.choice([0, 0, 1], B)]
    layer.step(nq, lens, 2, 20, pad=0)


@pytest.mark.parametrize("d,page", [(512, 64), (256, 256), (128, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_units_of_one_tile_and_runs_that_end_in_them(d, page, dtype):
    # few and many tiles a unit beside one another, so that runs begin and end at every place
    lens = [0, 1, 62, 63, 64, 127, 128, 129, 700, 5]
    layer = Layer(G.GLOBAL, 4, 2, d, 0, dtype, page, len(lens), -(-720 // page), 6)
    layer.step([max(1, c) if c else 1 for c in lens], [0] * len(lens), 1024, 0, pad=0)
    layer.step([1] * len(lens), [max(1, c) for c in lens], 1, 720, pad=0)
    layer.step([1] * len(lens), [max(1, c) + 1 for c in lens], 1, 1 << 20, pad=0)


def test_prefixes_that_decrease_are_recorded():
    layer = Layer(G.GLOBAL, 8, 1, 512, 0, "bf16", 64, 3, 4, 7)
    layer.step([6, 6, 6], [0, 0, 0], 8, 0, pad=0)
    q = torch.randn(8, 8, 512, device="cuda").to(torch.bfloat16)
    for max_q in (8, 200):
        out = torch.zeros(8, 8, 512, device="cuda")
        need = G.gemma_attn_paged_workspace_size(layer.p, layer.cache, 3, 8, max_q, 200)
        ws = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
        G.gemma_attn_paged_attend(layer.p, layer.cache, q, ints([0, 5, 3, 8]), ints([6, 6, 6]), out, None, 3, 8, max_q, 200, ws, need)
        with pytest.raises(G.GemmaAttnError) as e:
            G.gemma_attn_check()
        assert e.value.status == G.ERR_SEQLEN


def test_a_race_of_neighbouring_quotients():
    # quotients a few steps of fp32 apart, at every magnitude: what decides is the correctly rounded
    # quotient, then the index
    rng = np.random.default_rng(8)
    f, B, V = np.float32, 64, 5003
    top = rng.uniform(-140, 100, (B, 1))
    e = np.exp2(rng.uniform(-6, 6, (B, V))).astype(f)
    p = (e.astype(np.float64) * np.exp2(top) * (1 + rng.integers(-3, 4, (B, V)) * 2.0 ** -24)).astype(f)
    e[:, ::97] = np.array([0.0, -1.0, np.inf, np.nan], f)[rng.integers(0, 4, e[:, ::97].shape)]
    with np.errstate(all="ignore"):
        race = np.where((p > 0) & (e > 0), p / e, f(-1))
    want = np.where(np.isnan(race), f(-1), race).argmax(-1)
    acc, out = ints([9] * B), torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    G.gemma_attn_draft_verify(torch.tensor(p).view(B, 1, V).cuda(), None, torch.zeros(B, 0, dtype=torch.int32, device="cuda"), None,
                              torch.zeros(B, 0, device="cuda"), torch.tensor(e).cuda(), acc, out)
    assert acc.tolist() == [0] * B and out[:, 0].tolist() == want.tolist()


def test_more_kv_heads_than_a_plan_cuts_units():
    # a chunk's units go over all KV heads at once; with this many none may be cut
    layer = Layer(G.GLOBAL, 600, 600, 64, 0, "bf16", 16, 1, 6, 9)
    layer.step([70], [0], 70, 0, pad=0)
