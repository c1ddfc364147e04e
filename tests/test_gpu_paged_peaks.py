"""Attention over a paged cache for rows whose weights differ by orders of magnitude: a sink key
above a long flat tail, and value rows of very different size.

Bounds. Sinks: those of the other paged-cache tests (max-abs 1e-2, relative RMS 5e-3), here for
every row by itself. With a tail that holds 11 to 99 percent of a row, a kernel that keeps the
tail's mass in the sum and loses 1 percent of its values is off by more.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

G = pytest.importorskip("global_interleaved_layers_b200")
from gpu_util import TOL_LSE, TOL_MAX_ABS, TOL_REL_RMS  # noqa: E402
from paged_util import Cache, attend64, quantise64, run_attend  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    G.gemma_attn_check()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_sink(kind, d, dtype, tokens, batch, n, sink, spread, low=10.0, top=20.0):
    """`batch` sequences over the same n cached rows, 8 heads of `tokens` new tokens each: row i has
    its sink's weight 2^low to 2^top times the tail's, whose logits are equal or have a deviation of
    `spread`. Values have the mean 0.5, the sink's -0.5."""
    page, heads = 256, 8
    gen = torch.Generator(device="cuda").manual_seed(d + n + tokens)
    local = kind == G.LOCAL
    par = G.params(kind, heads, 1, d, window=1 << 20 if local else 0, rope_p=0.0)
    par.out_dtype = G.OUT_F32
    rows = [torch.randn(n, d, generator=gen, device="cuda") + 0.5 for _ in range(2 if local else 1)]
    for x in rows:
        x[sink] -= 1.0
    k = rows[0]
    k[:, 0] = 0.0          # the first dimension carries the sink's score
    k[sink] = k[sink].clamp(-4, 4)
    k[sink, 0] = 4.0
    pools, scales, held = [], [], []
    for x in rows:
        x = x.to(torch.bfloat16)
        if dtype == "e4m3":
            y, s = quantise64(x.double())
            codes = (y / s).float().to(torch.float8_e4m3fn)
            pools.append(codes.view(n // page, 1, page, d))
            scales.append(s.float().reshape(n // page, 1, page).contiguous())
            held.append(y)
        else:
            pools.append(x.view(n // page, 1, page, d))
            scales.append(None)
            held.append(x.double())
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").expand(batch, -1).contiguous()
    cache = G.paged_cache(pools[0], pools[1] if local else None, table, k_scales=scales[0],
                          v_scales=scales[1] if local else None)
    ratio = torch.linspace(low, top, tokens * heads, device="cuda")
    q = torch.zeros(tokens * heads, d, device="cuda")
    q[:, 1:] = torch.randn(tokens * heads, d - 1, generator=gen, device="cuda") * spread
    q[:, 0] = ratio * math.log(2) / (4 * par.softmax_scale)
    q = q.to(torch.bfloat16)
    T = batch * tokens
    out = torch.empty(T, heads, d, device="cuda")
    lse = torch.empty(T, heads, device="cuda")
    cu, lens = ints([tokens * b for b in range(batch + 1)]), ints([n - tokens] * batch)
    need = G.gemma_attn_paged_workspace_size(par, cache, batch, T, tokens, n)
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
    G.gemma_attn_paged_attend(par, cache, q.view(tokens, heads, d).repeat(batch, 1, 1), cu, lens, out, lse, batch, T, tokens, n,
                              ws, need)
    G.gemma_attn_check()
    s = q.double() @ held[0].T * par.softmax_scale
    pos = torch.arange(n, device="cuda")
    last = n - tokens + torch.arange(tokens, device="cuda").repeat_interleave(heads)
    s = s.masked_fill(pos[None] > last[:, None], -math.inf)
    ref = torch.softmax(s, -1) @ held[-1]
    diff = out.view(batch, tokens * heads, d).double() - ref
    assert float(diff.abs().max()) <= TOL_MAX_ABS, diff.abs().amax((0, 2)).tolist()
    rms = diff.norm(dim=-1) / ref.norm(dim=-1)
    assert float(rms.max()) <= TOL_REL_RMS, rms.amax(0).tolist()
    assert float((lse.view(batch, -1).double() - torch.logsumexp(s, -1)).abs().max()) <= TOL_LSE
    return float(diff.abs().max()), float(rms.max())


# 148 sequences: a unit of work is a whole sequence; 3: it is cut over the processors
@pytest.mark.parametrize("batch", [148, 3])
@pytest.mark.parametrize("spread", [0.0, 0.45])
@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", [G.GLOBAL, G.LOCAL])
@pytest.mark.parametrize("d", [128, 256, 512])
def test_a_sink_and_a_long_tail(kind, d, dtype, tokens, spread, batch):
    check_sink(kind, d, dtype, tokens, batch, 32768, 5 if tokens == 1 else 20000, spread)


@pytest.mark.parametrize("spread", [0.0, 0.45])
@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("kind,d", [(G.GLOBAL, 512), (G.LOCAL, 128)])
def test_a_sink_and_a_very_long_tail(kind, d, tokens, spread):
    check_sink(kind, d, "e4m3", tokens, 148, 131072, 20000 if tokens == 1 else 5, spread)


# 64 dims: 1184 sequences, each with a warp of its own, or 3 that are cut
@pytest.mark.parametrize("batch", [1184, 3])
@pytest.mark.parametrize("spread", [0.0, 0.45])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", [G.GLOBAL, G.LOCAL])
def test_a_sink_and_a_quarter_of_a_million_keys_of_64_dims(kind, dtype, spread, batch):
    check_sink(kind, 64, dtype, 1, batch, 262144, 70, spread, low=20.0, top=25.5)


@pytest.mark.parametrize("nq", [1, 4, 20])
@pytest.mark.parametrize("d", [128, 256, 512])
def test_value_scales_that_differ_between_keys(d, nq):
    """e4m3 values whose scales span 2^120, in the kernel that keeps a weight as two e4m3 numbers and
    the value's scale 2^k in it: W = p 2^k, off by at most 2^-8 of itself or, at the bottom, 2^-13
    where the row's largest is at least 2^7: 2^-20 of that. Its 200 keys' codes are at most 448
    beside one of more than 224 (a row's scale is the smallest that holds it), so the second part
    is at most 200 x 2 x 2^-20 of the row's largest sum of p|v|. Scores: with no rotation a query
    element is exact or off by 2^-21 of the row's largest, under 16 here; over 512 dims of keys of
    mean magnitude 0.8, at the score scale of 1 / sqrt(512): under 2^-12.8 of a score, so a weight
    and the sum move apart by under 2^-11 of a weight."""
    par = G.params(G.LOCAL, 2, 1, d, window=4096, rope_p=0.0)
    cache = Cache(G, G.LOCAL, 1, d, 16, "e4m3", [200], seed=5)
    f = torch.ones(200, dtype=torch.float64)
    f[::3], f[1::5], f[7] = 2.0 ** -30, 2.0 ** 30, 2.0 ** -90
    for i in range(200):
        cache.scales["v"][int(cache.table[0, i // 16]), :, i % 16] *= float(f[i])
    q = 3 * torch.randn(nq, 2, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    out, lse = run_attend(G, cache, par, q, (nq,), (200 - nq,))
    v = cache.rows["v"][0] * f.cuda()[:, None, None]
    args = (200 - nq, 4096, 0, 1e4, par.softmax_scale, False)
    ref, ref_lse = attend64(q.double(), cache.rows["k"][0], v, *args)
    G.gemma_attn_check()
    size, _ = attend64(q.double(), cache.rows["k"][0], v.abs(), *args)
    most = (2.0 ** -8 + 2.0 ** -11) * size + 400 * 2.0 ** -20 * size.amax(-1, keepdim=True)
    assert bool(((out.double() - ref).abs() <= most).all())
    assert float((lse.double() - ref_lse).abs().max()) <= TOL_LSE
