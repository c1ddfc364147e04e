"""Attend calls that follow one another without a pause over one workspace, their lengths and rows
rewritten on the device in between: every call's result is the one that it has alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu

G = pytest.importorskip("global_interleaved_layers_b200")
from paged_util import Cache  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    G.gemma_attn_check()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,hq,hkv,d,window", [(G.GLOBAL, 8, 1, 512, 0), (G.LOCAL, 8, 4, 256, 90), (G.GLOBAL, 4, 2, 64, 0)])
def test_calls_without_a_pause_over_one_workspace(kind, hq, hkv, d, window, dtype):
    par = G.params(kind, hq, hkv, d, window=window, rope_p=1.0 if kind == G.LOCAL else 0.25)
    B, T, max_len = 3, 400, 3000
    cache = Cache(G, kind, hkv, d, 32, dtype, [max_len + T] * B, seed=3)
    # plans that differ in everything: long chunks, a mixture, single tokens, nothing, other orders
    steps = [((300, 1, 99), (2000, 17, 0)), ((1, 1, 1), (2999, 5, 700)), ((0, 400, 0), (1, 3000, 9)), ((2, 0, 398), (33, 8, 129)),
             ((0, 0, 0), (5, 5, 5)), ((130, 135, 135), (1, 64, 2500))]
    steps = steps + steps[::-1] + [steps[i] for i in (2, 0, 4, 1, 5, 3)]
    gen = torch.Generator(device="cuda").manual_seed(1)
    plan = []
    for nq, ctx in steps:
        cu = [0, nq[0], nq[0] + nq[1], sum(nq)]
        plan.append((ints(cu), ints(ctx), torch.randn(T, hq, d, generator=gen, device="cuda").to(torch.bfloat16)))
    need = G.gemma_attn_paged_workspace_size(par, cache.handle, B, T, T, max_len)
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")

    def call(cu, lens, q, out, lse):
        G.gemma_attn_paged_attend(par, cache.handle, q, cu, lens, out, lse, B, T, T, max_len, ws, need)

    alone = []
    for cu, lens, q in plan:
        out, lse = torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, hq, device="cuda")
        torch.cuda.synchronize()
        call(cu, lens, q, out, lse)
        torch.cuda.synchronize()
        alone.append((out, lse))
    G.gemma_attn_check()
    cu, lens, q = (x.clone() for x in plan[0])
    for _ in range(3):
        got = [(torch.zeros_like(o), torch.zeros_like(s)) for o, s in alone]
        torch.cuda.synchronize()
        for (c, n, x), (out, lse) in zip(plan, got):
            q.copy_(x)
            lens.copy_(n)
            cu.copy_(c)
            call(cu, lens, q, out, lse)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(alone, got)):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), i
    G.gemma_attn_check()
