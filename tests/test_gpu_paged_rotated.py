"""Rotated rows of the kernel that serves 64 dims and K=V layers with many rotated pairs."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

G = pytest.importorskip("global_interleaved_layers_b200")
from paged_util import Cache, run_attend, turn64  # noqa: E402
from test_gpu_paged import check_attend  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    G.gemma_attn_check()


@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("dtype,half_step", [("bf16", 2.0 ** -8), ("e4m3", 2.0 ** -11)])
def test_a_rotated_query_is_rounded_once(dtype, half_step, tokens):
    """With a window of one key the log-sum-exp is the score. A head's query has one pair of
    dimensions, so that its two roundings (bf16 over bf16 pages; over e4m3 pages fp16, 2^-11 of a
    value at most) show in full: the score is off by that share of scale sum |q_i k_i|. Beside it
    the angle (2^-21 of |q| |k|), the fp32 products and the logarithm: 2^-18 of the same, and 2^-20."""
    d, hq, B = 64, 8, 48
    ctx = [int(x) for x in np.random.default_rng(4).integers(0, 3000, B)]
    par = G.params(G.LOCAL, hq, 1, d, window=1, rope_p=1.0, rope_base=1e4)
    cache = Cache(G, G.LOCAL, 1, d, 16, dtype, [c + tokens for c in ctx], seed=2, keep=list(ctx))
    gen = torch.Generator().manual_seed(7)
    q = torch.zeros(B * tokens, hq, d)
    for h in range(hq):
        for j in (4 * h, 4 * h + d // 2):
            q[:, h, j] = 30 * torch.randn(B * tokens, generator=gen)
    q = q.to(torch.bfloat16)
    out, lse = run_attend(G, cache, par, q.cuda(), [tokens] * B, ctx)
    G.gemma_attn_check()
    pos = torch.cat([torch.arange(c, c + tokens) for c in ctx])
    k = torch.cat([cache.rows["k"][b][c:c + tokens] for b, c in enumerate(ctx)]).cpu()
    turned = turn64(q.double(), pos, d // 2, 1e4)
    ref = (turned * k).sum(-1) * par.softmax_scale
    size = (turned * k).abs().sum(-1) * par.softmax_scale
    length = turned.norm(dim=-1) * k.norm(dim=-1) * par.softmax_scale
    most = half_step * size + 2.0 ** -18 * length + 2.0 ** -20
    assert bool(((lse.cpu().double() - ref).abs() <= most).all()), float(((lse.cpu().double() - ref).abs() / most).max())
    v = torch.cat([cache.rows["v"][b][c:c + tokens] for b, c in enumerate(ctx)])
    # one key: its value row comes back, to the quotient's rounding
    assert float((out.double() - v).abs().max()) <= 2.0 ** -20 * float(v.abs().max())


# more than 64 rotated pairs: one sequence, and so many that every warp has one of its own
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,p", [(256, 0.6), (256, 1.0), (512, 0.3), (512, 0.7), (512, 1.0)])
def test_many_rotated_pairs(d, p, dtype):
    check_attend(G.GLOBAL, 2, 1, d, 16, dtype, (1, 4, 0, 30), (300, 70, 5, 41), p=p)
    check_attend(G.GLOBAL, 8, 1, d, 32, dtype, (8, 1), (900, 2000), p=p)
    if d == 256:
        check_attend(G.GLOBAL, 8, 4, d, 16, dtype, (1,) * 150, [7 * i % 90 for i in range(150)], p=p)
