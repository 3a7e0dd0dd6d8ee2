"""How the cache calls' kernels read what the kernel in front of them wrote
(CPU, on the source).  They are resident while that kernel ends, so nothing
may be read as memory that is constant for the kernel's life, and the wait
stands in front of everything that is read."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_drafter_k3_gb300",
                    "csrc")
SOURCES = ["cache_common.cuh", "chunk_plan.cuh", "k3da_cache.cu", "k3da_chunk.cu", "k3da_chunk_small.cu", "sm103.cuh"]


def read(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", SOURCES)
def test_nothing_is_read_as_constant(name):
    src = read(name)
    for word in ("__ldg", "__ldca", "__ldcg", "__ldcs", "__ldlu", "__restrict__", ".nc."):
        assert word not in src, word


def test_loads_keep_their_place():
    src = read("cache_common.cuh")
    assert len(re.findall(r'asm volatile\("ld\.global\.', src)) == len(re.findall(r"ld\.global", src)) == 2


@pytest.mark.parametrize("name", ["k3da_cache.cu", "k3da_chunk.cu", "k3da_chunk_small.cu"])
def test_the_wait_comes_first(name):
    """In every kernel: no call argument that points to memory is used in
    front of its first wait_for_stream()."""
    src = read(name)
    kernels = [m.start() for m in re.finditer(r"__global__", src)]
    assert kernels
    for at in kernels:
        wait = src.index("wait_for_stream();", at)
        front = src[src.index("{", src.index("(const __grid_constant__", at)):wait]
        assert not re.search(r"p\.(qkv|pool|scales|page_table|ctx_lens|starts|cu_seqlens|positions|q_w|k_w|cuts|part_ml|part_o|"
                             r"out|lse|k_out|v_out|q_out)\b|\bp\.q\b|load_here|build_plan|tma_load|bulk_load", front), name
