"""The status word is written too: it may lie in nothing else that a call is
given (CPU: every call made here is refused)."""
import pytest

import speculative_decoding_drafter_k3_gb300 as k3da
import test_cache_overlaps as cache
import test_draft_abi as draft
from speculative_decoding_drafter_k3_gb300 import build as kbuild


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return k3da.load_library()


@pytest.mark.parametrize("what", draft.CALLS)
def test_calls_around_the_drafts(lib, what):
    for other, size in draft.SIZES[what].items():
        if other != "status":
            for at in (0, size - 4 - size % 4):
                assert draft.call(lib, what, status=draft.CALLS[what][other] + at) == k3da.EINVAL, (other, at)


@pytest.mark.parametrize("what", ["append", "append_qknorm", "gather", "attn"])
def test_cache_calls(lib, what):
    written, read = cache.sizes(what, lib)
    size = {**written, **read}
    for other in size:
        if other != "status":
            for byte in (0, size[other] - 4):
                at = {name: (i + 1) << 44 for i, name in enumerate(size)}
                at["status"] = at[other] + byte
                assert cache.call(what, lib, at) == k3da.EINVAL, (other, byte)
