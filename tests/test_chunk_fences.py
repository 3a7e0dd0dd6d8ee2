"""The tcgen05 fence rule on the chunk attention's source (CPU only): the lint
of test_tcgen05_fences.py, told the names of this kernel's tensor-memory and
barrier helpers as well, with mutants that remove single fences."""
import os

import pytest

import test_tcgen05_fences as lint

SOURCE = os.path.join(lint.CSRC, "k3da_chunk.cu")


@pytest.fixture(autouse=True)
def names(monkeypatch):
    tmem = ("tmem_ld32", "tmem_ld16", "tmem_ld8", "tmem_st16", "tmem_st8", "tmem_wait_ld")
    monkeypatch.setattr(lint, "TC_CALLS", lint.TC_CALLS + tmem[:5])
    monkeypatch.setattr(lint, "TMEM_TOUCH", lint.TMEM_TOUCH + tmem)


def source():
    return open(SOURCE).read()


def test_the_kernel_follows_the_fence_rule():
    found = lint.lint_source(source(), "k3da_chunk.cu")
    assert not found, "\n".join(f"{f}:{ln}: rule {r}: {msg}" for f, ln, r, msg in found)


def test_the_lint_reads_the_kernel():
    text, _ = lint._strip(source())
    for name in ("mma_ss(", "mma_ts(", "mma_commit(", "tmem_ld32(", "tmem_st16(", "fence_after()", "fence_before()",
                 "mbar_wait(", "mbar_arrive("):
        assert name in text, name


MUTANTS = {
    "no_fence_after_s_full_wait": ("// No row of this warp's", "fence_after();", True, "A"),
    "no_fence_after_rescale_wait": ("// A row's two threads scale", "fence_after();", True, "A"),
    "no_fence_after_merge_wait": ("mbar_wait(bar_xch", "fence_after();", True, "A"),
    "no_fence_before_p_handover": ("mbar_arrive(pfull);\n            }",
                                   "fence_before();", False, "B"),
    "no_fence_before_o_free": ("mbar_arrive(bar_ofree + 8 * s)", "fence_before();", False, "B"),
    "no_fence_after_buffer_wait": ("mbar_wait(bar_bfree + 8 * buf", "fence_after();", True, "A"),
    "no_fence_after_p_full_wait": ("mbar_wait(bar_pfull + 8 * turn", "fence_after();", True, "A"),
    "no_fence_after_final_barrier": ("tcgen05.dealloc", "fence_after();", False, "A"),
}


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_the_lint_catches_a_removed_fence(name):
    anchor, fence, after, rule = MUTANTS[name]
    bad = lint.lint_source(lint._remove(source(), anchor, fence, after))
    assert any(r == rule for _, _, r, _ in bad), name
