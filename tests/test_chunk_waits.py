"""The chunk attention's waits give up as a warp (CPU, on the source): where
one runs out, lanes that took answers of their own would come to the warp's
next operation apart, and hang there.  Nothing here can be made to happen on a
GPU that is to go on working, so the rule is read out of the source: a wait is
inside a vote, or in a lane's own branch, or in a loop that holds no operation
of the whole warp and has a vote behind it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_drafter_k3_gb300",
                    "csrc")
WARP_WIDE = r"__syncwarp|__shfl\w*|__any_sync|__all_sync|__ballot\w*|__reduce\w*|\bagreed\b|tmem_\w+|__syncthreads|elect_one"


def read(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def span(src, at, opening, closing):
    """From the bracket at or behind `at` to behind its partner."""
    i = src.index(opening, at)
    depth = 0
    for j in range(i, len(src)):
        depth += (src[j] == opening) - (src[j] == closing)
        if depth == 0:
            return i, j + 1
    raise ValueError("unbalanced")


def spans(src, head, opening, closing):
    return [span(src, m.end() - 1, opening, closing) for m in re.finditer(head, src)]


def waits_outside(src):
    """The waits that no rule covers (as source lines)."""
    good = spans(src, r"\bagreed\(", "(", ")") + spans(src, r"\b__all_sync\(", "(", ")")
    good += spans(src, r"if \(lane == 0\) \{", "{", "}")
    for a, b in spans(src, r"for \(int t = t0; t < t1; \+\+t\) \{", "{", "}"):
        if not re.search(WARP_WIDE, src[a:b]) and re.match(r"\s*alive = agreed\(alive\);\s*if \(!alive\) break;", src[b:]):
            good.append((a, b))
    lines = []
    for m in re.finditer(r"\bmbar_wait\(", src):
        if not any(a <= m.start() < b for a, b in good):
            lines.append(src[m.start():src.index("\n", m.start())])
    return lines


@pytest.mark.parametrize("name,number", [("k3da_chunk.cu", 19), ("k3da_chunk_small.cu", 1)])
def test_a_warp_gives_up_together(name, number):
    src = read(name)
    assert waits_outside(src) == []
    assert len(re.findall(r"\bmbar_wait\(", src)) >= number


def test_the_vote_is_a_vote():
    assert "bool agreed(bool mine) { return __all_sync(kFull, mine); }" in read("k3da_chunk.cu")


@pytest.mark.parametrize("bar", ["bar_sfull + 8", "bar_piece + 8", "bar_xch", "bar_rempty : part", "bar_vfull + 8"])
def test_a_missing_vote_is_seen(bar):
    src = read("k3da_chunk.cu")
    i = next(m.start() for m in re.finditer(r"agreed\(mbar_wait\(", src) if bar in src[m.start():m.start() + 60])
    assert waits_outside(src[:i] + "given(" + src[i + len("agreed("):])


def test_a_missing_vote_behind_the_products_is_seen():
    src = read("k3da_chunk.cu")
    assert waits_outside(src.replace("alive = agreed(alive);", ""))
    at = src.index("for (int t = t0; t < t1; ++t) {", src.index("next += step") - 3000)
    i, _ = span(src, at, "{", "}")
    assert waits_outside(src[:i + 1] + " __syncwarp(); " + src[i + 1:])


def test_loads_land_whatever_gives_up_when():
    """A copy that is still on its way must not outlive its CTA, also where a
    warp gives up after the one that issued the copy is done: what waits for
    the last copies stands behind the issuers' loops, under no condition on
    who gave up so far."""
    src = read("k3da_chunk.cu")
    assert "if (*abort_flag)" not in src and "if (!alive) {" not in src
    scheduler = src[src.index("Walk walk;"):src.index("const int u = warp >> 2")]
    tail = scheduler[scheduler.index("p.cuts[blockIdx.x] = cut;"):]
    assert re.search(r"for \(int s = 0; s < 2; \+\+s\) \{[^{}]*if \(n_fills > 0\) land\(bar_qfull", tail)
    a, b = span(src, src.index("for (int n = 0; alive; ++n) {", src.index("int issued[2]")), "{", "}")
    behind = src[b:src.index("} else if (warp < kPrepWarp)")]
    assert "land_ring(QUANT ? bar_rfull : bar_kfull" in behind and "if (!QUANT) land_ring(bar_vfull" in behind
    small = read("k3da_chunk_small.cu")
    a, b = span(small, small.index("for (int n = 0;; ++n) {", small.index("load.begin(warp")), "{", "}")
    assert small[b:].lstrip().startswith("load.drain();")
