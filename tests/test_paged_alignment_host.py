"""Lengths, prefixes and log-sum-exps that are not 4-byte aligned are refused before any launch."""
import pytest

G = pytest.importorskip("global_interleaved_layers_b200")

FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_words_are_refused(off):
    p = G.params(G.GLOBAL, 8, 1, 512, rope_p=0.25)
    c = G.GemmaAttnPagedCache(FAKE, None, None, None, FAKE, 10, 16, 4, G.PAGES_BF16)
    for f, args, words in [(G.gemma_attn_paged_append, [FAKE, None, FAKE, FAKE, 1, 4], (2, 3)),
                           (G.gemma_attn_paged_gather, [FAKE, FAKE, FAKE, None, 1, 4], (0, 1)),
                           (G.gemma_attn_paged_attend, [FAKE, FAKE, FAKE, FAKE, FAKE, 1, 4, 4, 16, FAKE, 1 << 40], (1, 2, 4))]:
        for at in words:
            bad = list(args)
            bad[at] = FAKE + off
            with pytest.raises(G.GemmaAttnError) as e:
                f(p, c, *bad, 0)
            assert e.value.status == G.ERR_MISALIGNED
    assert G.gemma_attn_last_launch_count() == 0
