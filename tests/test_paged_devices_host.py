"""Paged-cache and draft calls with tensors that no kernel can read are refused before the library
is called."""
import pytest
import torch

G = pytest.importorskip("global_interleaved_layers_b200")

bf, i32 = torch.bfloat16, torch.int32


class NoLibrary:
    def __getattr__(self, name):
        def called(*args):
            raise AssertionError(f"{name} was called")
        return called


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    error_string = G._lib.gemma_attn_error_string
    stub = NoLibrary()
    stub.gemma_attn_error_string = error_string
    monkeypatch.setattr(G, "_lib", stub)


def refused(f, *args):
    with pytest.raises(G.GemmaAttnError) as e:
        f(*args)
    assert e.value.status == G.ERR_INVALID_ARG and "CUDA" in str(e.value)


def calls(device, handle):
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
    p = G.params(G.GLOBAL, 4, 2, 64, rope_p=0.25)
    if handle == "tensors":
        c = G.paged_cache(z(6, 2, 16, 64), None, z(2, 3, dt=i32))
    else:
        c = G.GemmaAttnPagedCache(1 << 20, None, None, None, 1 << 20, 6, 16, 3, G.PAGES_BF16)
    cu, lens, ws = z(3, dt=i32), z(2, dt=i32), z(256, dt=torch.uint8)
    yield G.gemma_attn_paged_append, p, c, z(4, 2, 64), None, cu, lens, 2, 4
    yield G.gemma_attn_paged_gather, p, c, lens, cu, z(4, 2, 64), None, 2, 4
    yield G.gemma_attn_paged_attend, p, c, z(4, 4, 64), cu, lens, z(4, 4, 64), None, 2, 4, 2, 16, ws, 256
    yield G.gemma_attn_paged_attend, p, c, z(4, 4, 64), cu, lens, z(4, 4, 64), z(4, 4, dt=torch.float32), 2, 4, 2, 16, None, 0


@pytest.mark.parametrize("stream", [None, 0])
@pytest.mark.parametrize("handle", ["tensors", "addresses"])
@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_paged_calls_refuse_host_tensors(device, handle, stream):
    for f, *args in calls(device, handle):
        refused(f, *args, stream)


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_one_host_tensor_among_addresses_is_refused(device):
    for f, *args in calls(device, "addresses"):
        for keep in range(len(args)):
            if not isinstance(args[keep], torch.Tensor):
                continue
            refused(f, *[1 << 20 if isinstance(a, torch.Tensor) and i != keep else a for i, a in enumerate(args)])


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_draft_verification_refuses_host_tensors(device):
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
    refused(G.gemma_attn_draft_verify, z(2, 4, 9), z(2, 3, 9), z(2, 3, dt=i32), None, z(2, 3), z(2, 9), z(2, dt=i32), z(2, 4, dt=i32))
    refused(G.gemma_attn_draft_verify, z(2, 4, 9, dt=bf), None, z(2, 3, dt=i32), z(2, dt=i32), z(2, 3), z(2, 9), z(2, dt=i32),
            z(2, 4, dt=i32), 0)
