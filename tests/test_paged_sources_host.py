"""Rules of the paged-cache kernels' sources that no run can show."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "global_interleaved_layers_b200", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", ["paged_decode.cu", "paged_tile.cu", "paged_chunk.cu"])
def test_followers_read_nothing_through_the_read_only_path(name):
    # Blocks of these kernels are resident while the kernels before them still write the plan and
    # the inputs; ld.global.nc wants data that nothing writes while the kernel lives.
    text = code(name) + code("paged.h")
    assert not re.findall(r"\b__ldg\s*\(|ld\.global\.(?:\w+\.)*nc\b|__restrict__", text)


@pytest.mark.parametrize("name", ["paged_decode.cu", "paged_tile.cu", "paged_chunk.cu"])
def test_followers_wait_before_anything_else(name):
    # every kernel that launch_follower (or the chunk kernel's own launch) starts calls follow()
    # ahead of its first access to global memory: here, ahead of every load, store and atomic
    text = code(name)
    kernels = list(re.finditer(r"__global__[^{;]*?(\w+_kernel)\s*\([^{]*\)\s*\{", text))
    assert kernels
    for k in kernels:
        body = text[k.end():]
        first = body.index("follow();")
        assert not re.search(r"fresh\(|__ld|\ba\.\w+\[|\bp\.\w+\[|atomic|mbar_|tmem_|->", body[:first]), k.group(1)
