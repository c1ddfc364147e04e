"""Draft verification on the GPU, against the same rule written out in numpy, element by element.

Every operation of the rule is one correctly rounded fp32 operation, so results are equal."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

G = pytest.importorskip("global_interleaved_layers_b200")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    G.gemma_attn_check()


def rule(target, draft, tokens, lens, u, noise):
    B, n1, V = target.shape
    accepted, out = np.zeros(B, np.int32), np.full((B, n1), -1, np.int32)
    f = np.float32
    for b in range(B):
        n = n1 - 1 if lens is None else int(lens[b])
        i = 0
        while i < n:
            x = int(tokens[b, i])
            if not 0 <= x < V or not f(u[b, i]) * (f(1) if draft is None else f(draft[b, i, x])) < target[b, i, x]:
                break
            i += 1
        p = target[b, i]
        w = p.copy()
        if i < n:
            if draft is None:
                if 0 <= tokens[b, i] < V:
                    w[tokens[b, i]] = 0
            else:
                w = p - draft[b, i]
        token = -1
        for cand in (w, p):
            with np.errstate(all="ignore"):
                race = np.where((cand > 0) & (noise[b] > 0), cand / noise[b], f(-1))
            race = np.where(np.isnan(race), f(-1), race)
            if race.max() >= 0:
                token = int(race.argmax())  # the first of a tie
                break
        accepted[b] = i
        out[b, :i] = tokens[b, :i]
        out[b, i] = token
    return accepted, out


def run(target, draft, tokens, lens, u, noise):
    c = lambda x: None if x is None else torch.as_tensor(x).cuda().contiguous()  # noqa: E731
    B, n1, _ = target.shape
    acc = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    out = torch.full((B, n1), 77, dtype=torch.int32, device="cuda")
    G.gemma_attn_draft_verify(c(target), c(draft), c(tokens), c(lens), c(u), c(noise), acc, out)
    assert G.gemma_attn_last_launch_count() == 1
    return acc.cpu().numpy(), out.cpu().numpy()


def inputs(B, n, V, seed, near=0.5):
    r = np.random.default_rng(seed)
    logits = r.standard_normal((B, n + 1, V)).astype(np.float32) * 2

    def soft(z):
        e = np.exp(z - z.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)

    t = soft(logits)
    d = soft(logits[:, :n] + near * r.standard_normal((B, n, V)).astype(np.float32))
    tokens = np.array([[r.choice(V, p=d[b, i].astype(np.float64) / d[b, i].astype(np.float64).sum()) for i in range(n)]
                       for b in range(B)], np.int32).reshape(B, n)
    return t, d, tokens, r.random((B, n)).astype(np.float32), r.standard_exponential((B, V)).astype(np.float32)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (1, 4, 2), (3, 5, 31), (7, 3, 4097), (2, 8, 50001), (40, 2, 1024), (1, 0, 333), (2, 40, 65)])
def test_against_the_rule(B, n, V, certain, bf16):
    for seed in range(3):
        t, d, tokens, u, noise = inputs(B, n, V, 10 * seed + V)
        if bf16:
            t, d = torch.from_numpy(t).to(torch.bfloat16), torch.from_numpy(d).to(torch.bfloat16)
            ref = (t.float().numpy(), None if certain else d.float().numpy())
        else:
            ref = (t, None if certain else d)
        lens = None if seed == 0 else np.random.default_rng(seed).integers(0, n + 1, B).astype(np.int32)
        got = run(t, None if certain else d, tokens, lens, u, noise)
        want = rule(ref[0], ref[1], tokens, lens, u, noise)
        np.testing.assert_array_equal(got[0], want[0])
        np.testing.assert_array_equal(got[1], want[1])
    G.gemma_attn_check()


def test_ties_go_to_the_lowest_index():
    for V in (9, 20000):
        t = np.full((1, 1, V), 0.5, np.float32)
        noise = np.full((1, V), 2.0, np.float32)
        t[0, 0, :5] = 0
        none, uni = np.zeros((1, 0), np.int32), np.zeros((1, 0), np.float32)
        got = run(t, np.zeros((1, 0, V), np.float32), none, None, uni, noise)
        assert got[1].tolist() == [[5]]


def test_edges_of_the_rule():
    V = 1000
    t, d, tokens, u, noise = inputs(6, 2, V, 5)
    t[0, 0, tokens[0, 0]] = 0                     # p(x) = 0 is never accepted, not even at u = 0
    u[0, 0] = 0
    d[1, 0, tokens[1, 0]] = 0                     # q(x) = 0 < p(x) always is
    u[1, 0] = np.nextafter(np.float32(1), np.float32(0))
    t[2] = d[2, :1]                               # p = q everywhere, rejected by u = 1: no residual, p itself
    u[2, :] = 1.0
    t[3, 0] = 0                                   # nothing to draw from: -1
    noise[4, ::2] = 0                             # entries that are not positive never win
    noise[4, 1] = np.nan
    tokens[5, 0] = V                              # outside the vocabulary
    got, want = run(t, d, tokens, None, u, noise), rule(t, d, tokens, None, u, noise)
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])
    assert got[0][0] == 0 and got[0][1] >= 1 and got[0][2] == 0 and got[1][2, 0] >= 0 and got[1][3, 0] == -1
    assert got[1][4, got[0][4]] % 2 == 1 and got[0][5] == 0
    G.gemma_attn_check()


def test_lengths_out_of_range_are_brought_in_and_recorded():
    t, d, tokens, u, noise = inputs(2, 3, 100, 8)
    got = run(t, d, tokens, np.array([9, -2], np.int32), u, noise)
    with pytest.raises(G.GemmaAttnError) as e:
        G.gemma_attn_check()
    assert e.value.status == G.ERR_SEQLEN
    want = rule(t, d, tokens, np.array([3, 0]), u, noise)
    np.testing.assert_array_equal(got[0], want[0])
    np.testing.assert_array_equal(got[1], want[1])


def test_the_draw_follows_the_residual():
    """Accept-or-replace leaves the target's distribution: over many rounds the first token's
    frequencies are the target's. 40,000 rounds: a frequency's standard deviation is at most
    sqrt(p / 40000); five of them bound every one of 8 tokens (a false alarm in 200,000 seeds)."""
    V, B = 8, 40000
    r = np.random.default_rng(11)
    p, q = r.dirichlet(np.ones(V)).astype(np.float32), r.dirichlet(np.ones(V)).astype(np.float32)
    tokens = r.choice(V, size=(B, 1), p=q.astype(np.float64) / q.astype(np.float64).sum()).astype(np.int32)
    t, d = np.broadcast_to(p, (B, 2, V)), np.broadcast_to(q, (B, 1, V))
    _, out = run(np.ascontiguousarray(t), np.ascontiguousarray(d), tokens, None, r.random((B, 1)).astype(np.float32),
                 r.standard_exponential((B, V)).astype(np.float32))
    freq = np.bincount(out[:, 0], minlength=V) / B
    assert np.all(np.abs(freq - p) <= 5 * np.sqrt(p / B))
