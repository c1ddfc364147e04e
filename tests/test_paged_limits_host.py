"""Limits and names of the paged-cache entry points that need no GPU."""
import ctypes

import pytest

G = pytest.importorskip("global_interleaved_layers_b200")


def test_the_page_status_has_a_name():
    assert G.ERR_PAGE == -9
    text = G.gemma_attn_error_string(G.ERR_PAGE)
    assert "page" in text


@pytest.mark.parametrize("kind,d,hkv", [(G.GLOBAL, 64, 8), (G.GLOBAL, 512, 32)])
def test_a_batch_with_too_many_blocks_of_keys_is_refused(kind, d, hkv):
    # blocks of 16 keys (64 dims) or tiles of 64: batch x KV heads x blocks from 2^31 on
    p = G.params(kind, hkv, hkv, d, rope_p=0.25)
    per = 16 if d == 64 else 64
    cache = G.GemmaAttnPagedCache(1 << 20, None, None, None, 1 << 20, 1000, 256, 1 << 20, G.PAGES_BF16)
    keys = (1 << 31) // (60000 * hkv) * per
    with pytest.raises(G.GemmaAttnError) as e:
        G.gemma_attn_paged_workspace_size(p, cache, 60000, 60000, 1, keys)
    assert e.value.status == G.ERR_UNSUPPORTED
    assert G.gemma_attn_paged_workspace_size(p, cache, 60000, 60000, 1, keys // 4) > 0


def test_vocabularies_past_the_index_range_are_refused():
    f = 1 << 20  # never dereferenced: the check comes first
    args = [f, f, G.PROBS_F32, f, ctypes.c_void_p(None), f, f, 2, 3, (1 << 30) + 1, f, f, 0]
    assert G.raw_call("gemma_attn_draft_verify", *args) == G.ERR_UNSUPPORTED
