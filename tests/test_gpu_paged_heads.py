"""Large groups of query heads over one KV head: up to the 128 that are allowed, where one token
is a chunk of its own, and the sizes around the borders of the kernels' units."""
import pytest
import torch

pytestmark = pytest.mark.gpu

G = pytest.importorskip("global_interleaved_layers_b200")
from test_gpu_paged import check_attend  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    G.gemma_attn_check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,d,window", [(G.GLOBAL, 512, 0), (G.LOCAL, 256, 70), (G.LOCAL, 128, 1000), (G.GLOBAL, 64, 0)])
@pytest.mark.parametrize("group", [9, 33, 41, 64, 65, 100, 128])
def test_groups_of_many_heads(group, kind, d, window, dtype):
    check_attend(kind, 2 * group, 2, d, 32, dtype, (1, 0, 1, 1), (0, 9, 130, 700), window, pad_rows=2)
    check_attend(kind, group, 1, d, 64, dtype, (2, 1, 3), (63, 300, 0), window)
