"""Rows of zeros among small ones over e4m3 pages. A row of zeros is stored with the scale 1, far
above the scales of small rows; it adds nothing to an output and must not cost the others bits.

Bounds, per element, as for value scales that differ between keys: a weight times its value row's
scale is off by at most 2^-8 of itself or 2^-20 of the largest among the rows that are not zero. The 200
keys' codes are at most 448 beside one of more than 224: the second part is at most 200 x 2 x 2^-20 of
the row's largest sum of p|v|. Scores move a weight by under 2^-11 of itself."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

G = pytest.importorskip("global_interleaved_layers_b200")
from gpu_util import TOL_LSE  # noqa: E402
from paged_util import attend64, quantise64  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    G.gemma_attn_check()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("size", [1.0, 2.0 ** -12, 2.0 ** -34])
@pytest.mark.parametrize("nq", [1, 4, 20])
@pytest.mark.parametrize("kind", [G.LOCAL, G.GLOBAL])
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_rows_of_zeros_cost_the_others_nothing(d, kind, nq, size):
    n, page, local = 200, 16, kind == G.LOCAL
    gen = torch.Generator().manual_seed(d + nq)
    par = G.params(kind, 2, 1, d, window=4096 if local else 0, rope_p=0.0)
    par.out_dtype = G.OUT_F32
    zero = torch.zeros(n, dtype=torch.bool)
    zero[::3] = True
    zero[n - nq - 1] = zero[150:166] = True          # a page of nothing else among them
    k = torch.randn(n, 1, d, generator=gen)
    v = size * torch.randn(n, 1, d, generator=gen)
    v[zero] = 0.0
    v[zero.nonzero()[1], 0, ::2] = -0.0
    if local:
        k[3] = 2.0 * k[3].abs()                      # (a row of zeros) and queries that like it
    else:
        k = v
    q = torch.randn(nq, 2, d, generator=gen) + (0.5 if local else 0.0)
    k, v, q = (x.to(torch.bfloat16) for x in (k, v, q))
    blocks = -(-n // page)
    table = torch.randperm(blocks, generator=gen).to(torch.int32).view(1, blocks).cuda()
    pool = lambda: torch.full((blocks, 1, page, d), math.nan).to(torch.float8_e4m3fn).cuda()  # noqa: E731
    scales = [torch.full((blocks, 1, page), math.nan, device="cuda") for _ in range(2)]
    cache = G.paged_cache(pool(), pool() if local else None, table, k_scales=scales[0], v_scales=scales[1] if local else None)
    G.gemma_attn_paged_append(par, cache, k.cuda(), v.cuda() if local else None, ints([0, n]), ints([0]), 1, n)
    at = lambda i: (int(table[0, i // page]), 0, i % page)  # noqa: E731
    assert all(float(scales[1 if local else 0][at(int(i))]) == 1.0 for i in zero.nonzero())
    out, lse = torch.empty(nq, 2, d, device="cuda"), torch.empty(nq, 2, device="cuda")
    need = G.gemma_attn_paged_workspace_size(par, cache, 1, nq, nq, n)
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
    G.gemma_attn_paged_attend(par, cache, q.cuda(), ints([0, nq]), ints([n - nq]), out, lse, 1, nq, nq, n, ws, need)
    G.gemma_attn_check()
    kk, vv = quantise64(k.double())[0], quantise64(v.double())[0]
    args = (n - nq, 4096 if local else 0, 0, 1e4, par.softmax_scale, False)
    ref, ref_lse = attend64(q.double(), kk, vv, *args)
    mass, _ = attend64(q.double(), kk, vv.abs(), *args)
    most = (2.0 ** -8 + 2.0 ** -11) * mass + 400 * 2.0 ** -20 * mass.amax(-1, keepdim=True)
    off = (out.cpu().double() - ref).abs() / most
    assert float(off.max()) <= 1.0, float(off.max())
    assert float((lse.cpu().double() - ref_lse).abs().max()) <= TOL_LSE
