"""What the combine kernel takes from the CTAs before it (CPU): a cut that
names rows, CTAs or a head that there are not is left alone, and every way out
of the kernels leaves a cut.  (A wait that gives up must end as a status bit,
whatever the workspace held.)"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_drafter_k3_gb300", "csrc")

HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include "chunk_cut.h"
int main(int argc, char **argv) {
    for (int i = 1; i + 7 < argc; i += 8) {
        k3da_chunk::Cut cut = {};
        cut.has[1] = 1;
        cut.row = std::atoi(argv[i]);
        cut.tokens = std::atoi(argv[i + 1]);
        cut.head = std::atoi(argv[i + 2]);
        cut.last = std::atoi(argv[i + 3]);
        std::printf("%d\n", k3da_chunk::cut_fits(cut, std::atoi(argv[i + 4]), std::atoi(argv[i + 5]),
                                                 std::atoi(argv[i + 6]), std::atoi(argv[i + 7])));
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def fits(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("cuts")
    (d / "h.cpp").write_text(HARNESS)
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, str(d / "h.cpp"), "-o", str(d / "h")], check=True)

    def run(cases):
        args = [str(v) for c in cases for v in c]
        out = subprocess.run([str(d / "h")] + args, check=True, capture_output=True, text=True).stdout.split()
        return [x == "1" for x in out]
    return run


INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1
VALUES = {"row": [INT_MIN, -1, 0, 1, 99, 100, 101, INT_MAX], "tokens": [INT_MIN, -1, 0, 1, 42, 43, 100, 101, INT_MAX],
          "head": [INT_MIN, -1, 0, 3, 4, INT_MAX], "last": [INT_MIN, -1, 0, 6, 7, 8, 151, 152, INT_MAX]}


def test_every_cut_that_passes_is_in_bounds(fits):
    owner, rows, heads, most = 7, 100, 4, 42
    cases = [(r, t, h, l) for r in VALUES["row"] for t in VALUES["tokens"] for h in VALUES["head"] for l in VALUES["last"]]
    got = fits([c + (owner, rows, heads, most) for c in cases])
    want = [0 <= r and 0 <= t <= most and r + t <= rows and 0 <= h < heads and owner <= l < 152 for r, t, h, l in cases]
    assert got == want and any(got) and not all(got)


def test_the_combine_asks_before_it_indexes():
    src = open(os.path.join(CSRC, "k3da_chunk.cu")).read()
    body = src[src.index("k3da_chunk_combine_kernel(const"):]
    body = body[:body.index("// ---", 10)]
    asks = body.index("cut_fits(cut, a, p.T, p.Hkv, 2 * p.tpt)) return;")
    for use in ("cut.last - a", "cut.row + token", "cut.head * p.G", "continues[a + i]"):
        assert body.index(use) > asks, use


def test_every_way_out_of_a_kernel_leaves_a_cut():
    long, small = (open(os.path.join(CSRC, f)).read() for f in ("k3da_chunk.cu", "k3da_chunk_small.cu"))
    for src in (long, small):  # no items
        assert re.search(r"p\.cuts\[blockIdx\.x\] = Cut\{\};\s*wait_for_stream\(\);\s*return;", src)
    # The long chunks' scheduler: behind its loop, whatever ended that.
    loop = long[long.index("Walk walk;"):long.index("-- softmax --")]
    assert "\n            p.cuts[blockIdx.x] = cut;" in loop and "return" not in loop
    # The other's: with the end's mark, or where a wait gives up before it.
    loop = small[small.index("Walk walk;"):small.index("-- page warps --")]
    assert "if (!more) p.cuts[blockIdx.x] = cut;" in loop
    assert "return" not in loop
    for m in re.finditer(r"if \(!warp_wait\([^;]*?\)\)\s*(\{.*?\}|break;)", loop, re.S):
        assert "if (lane == 0 && more) p.cuts[blockIdx.x] = Cut{" in m.group(1)


PAGES_HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include "chunk_cut.h"
int main(int argc, char **argv) {
    for (int i = 1; i + 1 < argc; i += 2)
        std::printf("%d\n", k3da_chunk::page_masked(std::atoi(argv[i]), std::atoi(argv[i + 1])));
    return 0;
}
"""


def test_pages_at_the_end_of_the_longest_table(tmp_path):
    """In 32 bits, with overflows trapped: every page a tile can begin up to
    2^31 - 64 keys, against whole numbers."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    (tmp_path / "p.cpp").write_text(PAGES_HARNESS)
    subprocess.run([gxx, "-std=c++17", "-O0", "-ftrapv", "-I", CSRC, str(tmp_path / "p.cpp"), "-o", str(tmp_path / "p")], check=True)
    end = (2 ** 25 - 1) * 64
    pages = [0, 64, 128, end - 192, end - 128, end - 64, end]
    cases = [(p, n) for p in pages for q in pages for n in (q - 1, q, q + 1, q + 63, q + 64, q + 65) if 0 <= n <= end]
    out = subprocess.run([str(tmp_path / "p")] + [str(v) for c in cases for v in c], check=True, capture_output=True, text=True).stdout.split()
    assert out == ["1" if p + 64 > n else "0" for p, n in cases]
    for name in ("k3da_chunk.cu", "k3da_chunk_small.cu"):
        src = open(os.path.join(CSRC, name)).read()
        assert "page_masked(key0, least)" in src and "key0 + kP" not in src
