"""Refusals of the paged-cache and draft entry points: checked on the host, before any launch."""
import ctypes

import pytest
import torch

G = pytest.importorskip("global_interleaved_layers_b200")

FAKE = 1 << 20  # never dereferenced: validation fails first


def layer(kind=G.GLOBAL, hq=8, hkv=1, d=512, **kw):
    return G.params(kind, hq, hkv, d, window=64 if kind == G.LOCAL else 0, rope_p=0.25, **kw)


def cache(v=None, ks=None, vs=None, k=FAKE, table=FAKE, pages=10, ps=16, blocks=4, dtype=G.PAGES_BF16):
    return G.GemmaAttnPagedCache(k, v, ks, vs, table, pages, ps, blocks, dtype)


def status(f, *args):
    with pytest.raises(G.GemmaAttnError) as e:
        f(*args)
    return e.value.status


BAD_CACHES = [
    (layer(), cache(v=FAKE), G.ERR_INVALID_ARG),                       # a K=V layer with values
    (layer(G.LOCAL), cache(), G.ERR_INVALID_ARG),                      # a sliding-window layer without
    (layer(), cache(dtype=2), G.ERR_INVALID_ARG),
    (layer(), cache(ks=FAKE), G.ERR_INVALID_ARG),                      # bf16 with scales
    (layer(), cache(dtype=G.PAGES_E4M3), G.ERR_INVALID_ARG),           # e4m3 without
    (layer(G.LOCAL), cache(v=FAKE, ks=FAKE, dtype=G.PAGES_E4M3), G.ERR_INVALID_ARG),
    (layer(), cache(k=None), G.ERR_INVALID_ARG),
    (layer(), cache(table=None), G.ERR_INVALID_ARG),
    (layer(), cache(pages=0), G.ERR_INVALID_ARG),
    (layer(), cache(blocks=0), G.ERR_INVALID_ARG),
    (layer(), cache(ps=8), G.ERR_UNSUPPORTED),
    (layer(), cache(ps=48), G.ERR_UNSUPPORTED),
    (layer(), cache(ps=512), G.ERR_UNSUPPORTED),
    (layer(), cache(ps=0), G.ERR_UNSUPPORTED),
    (layer(), cache(k=FAKE + 8), G.ERR_MISALIGNED),
    (layer(), cache(ks=FAKE + 4, dtype=G.PAGES_E4M3), G.ERR_MISALIGNED),
    (layer(), cache(table=FAKE + 2), G.ERR_MISALIGNED),
    (layer(hq=32, hkv=16), cache(pages=1 << 28), G.ERR_UNSUPPORTED),
    (layer(d=32), cache(), G.ERR_UNSUPPORTED),
    (layer(d=96), cache(), G.ERR_UNSUPPORTED),
    (layer(hq=129), cache(), G.ERR_UNSUPPORTED),
    (layer(hq=9, hkv=2), cache(), G.ERR_INVALID_ARG),
    (G.params(G.BIDIR, 8, 8, 64), cache(v=FAKE), G.ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("i", range(len(BAD_CACHES)))
def test_bad_layers_and_caches(i):
    p, c, code = BAD_CACHES[i]
    v = FAKE if c.v_pages else None
    assert status(G.gemma_attn_paged_append, p, c, FAKE, v, FAKE, FAKE, 1, 4, 0) == code
    assert status(G.gemma_attn_paged_gather, p, c, FAKE, FAKE, FAKE, v, 1, 4, 0) == code
    assert status(G.gemma_attn_paged_workspace_size, p, c, 1, 4, 4, 16) == code
    assert status(G.gemma_attn_paged_attend, p, c, FAKE, FAKE, FAKE, FAKE, None, 1, 4, 4, 16, FAKE, 1 << 40, 0) == code
    assert G.gemma_attn_last_launch_count() == 0


def test_bad_arguments():
    p, c = layer(), cache()
    loc, lc = layer(G.LOCAL), cache(v=FAKE)
    bad, mis, uns = G.ERR_INVALID_ARG, G.ERR_MISALIGNED, G.ERR_UNSUPPORTED
    for args, code in [((FAKE, None, None, FAKE, 1, 4), bad), ((FAKE, None, FAKE, None, 1, 4), bad),
                       ((None, None, FAKE, FAKE, 1, 4), bad), ((FAKE, FAKE, FAKE, FAKE, 1, 4), bad),
                       ((FAKE, None, FAKE, FAKE, 0, 4), bad), ((FAKE, None, FAKE, FAKE, 1, -1), bad),
                       ((FAKE, None, FAKE, FAKE, 65536, 4), uns), ((FAKE + 2, None, FAKE, FAKE, 1, 4), mis)]:
        assert status(G.gemma_attn_paged_append, p, c, *args, 0) == code
    assert status(G.gemma_attn_paged_append, loc, lc, FAKE, None, FAKE, FAKE, 1, 4, 0) == bad
    for args, code in [((None, FAKE, FAKE, None, 1, 4), bad), ((FAKE, None, FAKE, None, 1, 4), bad),
                       ((FAKE, FAKE, None, None, 1, 4), bad), ((FAKE, FAKE, FAKE, FAKE, 1, 4), bad),
                       ((FAKE, FAKE, FAKE + 8, None, 1, 4), mis), ((FAKE, FAKE, FAKE, None, 1, -4), bad)]:
        assert status(G.gemma_attn_paged_gather, p, c, *args, 0) == code
    ok = [FAKE, FAKE, FAKE, FAKE, None, 1, 4, 4, 16, FAKE, 1 << 40]
    for at, value, code in [(0, None, bad), (1, None, bad), (2, None, bad), (3, None, bad), (0, FAKE + 2, mis), (3, FAKE + 4, mis),
                            (5, 0, bad), (5, 65536, uns), (6, -1, bad), (7, -1, bad), (8, -1, bad), (9, FAKE + 64, mis),
                            (8, 0x7fffffff, uns), (6, 0x7fffffff, uns)]:
        args = list(ok)
        args[at] = value
        assert status(G.gemma_attn_paged_attend, p, c, *args, 0) == code, (at, value)


def test_workspace_is_checked_against_its_size():
    p, c = layer(), cache(pages=4000, blocks=4000)
    need = G.gemma_attn_paged_workspace_size(p, c, 1, 1, 1, 60000)
    assert need > 0
    assert status(G.gemma_attn_paged_attend, p, c, FAKE, FAKE, FAKE, FAKE, None, 1, 1, 1, 60000, FAKE, need - 1, 0) == G.ERR_WORKSPACE
    assert status(G.gemma_attn_paged_attend, p, c, FAKE, FAKE, FAKE, FAKE, None, 1, 1, 1, 60000, None, need, 0) == G.ERR_WORKSPACE


def test_nothing_to_do_launches_nothing():
    p, c = layer(), cache()
    G.gemma_attn_paged_append(p, c, None, None, FAKE, FAKE, 3, 0, 0)
    G.gemma_attn_paged_gather(p, c, FAKE, FAKE, None, None, 3, 0, 0)
    G.gemma_attn_paged_attend(p, c, None, FAKE, FAKE, None, None, 3, 0, 0, 16, None, 0, 0)
    assert G.gemma_attn_last_launch_count() == 0


def test_bad_draft_arguments():
    ok = [FAKE, FAKE, G.PROBS_F32, FAKE, None, FAKE, FAKE, 2, 3, 100, FAKE, FAKE, 0]
    for at, value, code in [(0, None, -1), (2, 7, -1), (3, None, -1), (5, None, -1), (6, None, -1), (7, -1, -1), (8, -1, -1),
                            (9, 0, -1), (10, None, -1), (11, None, -1), (0, FAKE + 2, -4), (6, FAKE + 1, -4), (8, 1 << 21, -2)]:
        args = list(ok)
        args[at] = value
        assert G.raw_call("gemma_attn_draft_verify", *[ctypes.c_void_p(a) if a is None else a for a in args]) == code, (at, value)
    args = list(ok)
    args[7] = 0
    assert G.raw_call("gemma_attn_draft_verify", *args) == 0 and G.gemma_attn_last_launch_count() == 0


def test_tensors_are_checked_by_the_binding():
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(6, 2, 16, 64, dtype=bf)
    tab = torch.zeros(2, 3, dtype=i32)
    p = G.params(G.GLOBAL, 4, 2, 64, rope_p=0.25)
    c = G.paged_cache(k, None, tab)
    assert (c.num_pages, c.page_size, c.max_blocks, c.dtype) == (6, 16, 3, G.PAGES_BF16)
    for args, kw in [((k.float(), None, tab), {}), ((k.transpose(1, 2), None, tab), {}), ((k, k[:3], tab), {}), ((k, None, tab.long()), {}),
                     ((k, None, tab), {"k_scales": torch.zeros(6, 2, 16)}), ((k.to(torch.float8_e4m3fn), None, tab), {}),
                     ((k.to(torch.float8_e4m3fn), None, tab), {"k_scales": torch.zeros(6, 2, 15)}), ((k[0], None, tab), {})]:
        assert status(lambda: G.paged_cache(*args, **kw)) == G.ERR_INVALID_ARG
    new = torch.zeros(4, 2, 64, dtype=bf)
    cu, lens = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    for a in [(new.float(), None, cu, lens, 2, 4), (new, None, cu, lens, 2, 5), (new, None, cu[:2], lens, 2, 4),
              (new, None, cu, lens.long(), 2, 4), (new.expand(4, 2, 64)[:, :, ::2], None, cu, lens, 2, 4),
              (new, None, torch.zeros(4, dtype=i32), torch.zeros(3, dtype=i32), 3, 4)]:
        assert status(G.gemma_attn_paged_append, p, c, *a, 0) == G.ERR_INVALID_ARG
    assert status(G.gemma_attn_paged_append, G.params(G.GLOBAL, 4, 1, 64), c, new, None, cu, lens, 2, 4, 0) == G.ERR_INVALID_ARG
    q = torch.zeros(4, 4, 64, dtype=bf)
    ws = torch.zeros(256, dtype=torch.uint8)
    assert status(G.gemma_attn_paged_attend, p, c, q, cu, lens, q.float(), None, 2, 4, 2, 16, ws, 0, 0) == G.ERR_INVALID_ARG
    assert status(G.gemma_attn_paged_attend, p, c, q, cu, lens, q, None, 2, 4, 2, 16, ws, 257, 0) == G.ERR_INVALID_ARG
    t, d = torch.zeros(2, 4, 9), torch.zeros(2, 3, 9)
    tok, u, nz = torch.zeros(2, 3, dtype=i32), torch.zeros(2, 3), torch.zeros(2, 9)
    acc, out = torch.zeros(2, dtype=i32), torch.zeros(2, 4, dtype=i32)
    good = [t, d, tok, None, u, nz, acc, out]
    for at, x in [(0, t.double()), (1, d.to(bf)), (2, tok.long()), (3, torch.zeros(3, dtype=i32)), (4, u[:1]), (5, nz.t().contiguous().t()),
                  (6, acc.long()), (7, out[:, :3])]:
        args = list(good)
        args[at] = x
        assert status(G.gemma_attn_draft_verify, *args, 0) == G.ERR_INVALID_ARG
