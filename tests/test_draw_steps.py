"""How near a draw comes to the distribution that it draws from, by the
definition (CPU); and a drafter whose rows predict their own position (GPU)."""
import numpy as np
import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da
from draft_cases import draw, whole
from test_verify import Blocks, i32

STEPS = 2 ** 24


def shares(weights):
    """Of the 2^24 shares of a uniform number, how many draw each word."""
    run = np.concatenate([[0], np.cumsum(weights)])
    total = int(run[-1])
    first = [-(-int(c) * STEPS // total) for c in run]  # the first share whose place is at c or behind
    return np.diff(first)


@pytest.mark.parametrize("V,sharp", [(2, 1.0), (7, 3.0), (1000, 2.0), (20011, 4.0)])
def test_a_draw_is_off_by_less_than_a_step_a_word(V, sharp):
    """Each word's probability is met to 2^-24 (one step of the uniform number)
    and, of weights that add up to 1, V 2^-40 for what is cut off them; a word
    whose share of the total is above 2^-24 is always drawn by some number."""
    x = np.random.default_rng(V).normal(size=V) * sharp
    p = np.exp(x - x.max())
    p = (p / p.sum()).astype(np.float32)
    w = whole(p)
    n, exact = shares(w), p.astype(np.float64) / p.astype(np.float64).sum()
    assert n.sum() == STEPS
    assert (np.abs(n - w / w.sum() * STEPS) < 1).all()
    assert np.abs(n / STEPS - exact).max() < 2.0 ** -24 + V * 2.0 ** -40
    assert (n[w / w.sum() >= 2.0 ** -24] > 0).all()
    # They are the draws.
    at = np.cumsum(n)
    for k in np.flatnonzero(n)[:: max(1, (n > 0).sum() // 20)]:
        assert draw(w, (at[k] - 1) / STEPS) == draw(w, (at[k] - n[k]) / STEPS) == k


def test_words_below_a_step_may_never_be_drawn():
    """2^25 steps would be needed for all of these; half of them go without."""
    w = np.full(2 ** 12, 2 ** 15, np.int64)  # together 2^27
    w[0] = 2 ** 40 - 2 ** 27
    n = shares(w)
    assert set(n[1:].tolist()) <= {0, 1} and (n[1:] == 0).any()


@pytest.mark.gpu
@pytest.mark.parametrize("V", [41, 5003])
def test_a_drafter_whose_rows_predict_their_own_position(V):
    """Row i of such a drafter has the distribution of token i itself: its
    probabilities are passed from the second row on, out of one row more."""
    b = Blocks([6, 1, 0, 4, 3], V, 5)
    own = torch.full((b.T + 1, V), 7.0, device="cuda")
    own[1:] = b.q.cuda()
    out, num = torch.full((b.T,), -7, dtype=torch.int32, device="cuda"), i32([-9] * 5)
    k3da.k3da_verify(out, num, b.tokens.int().cuda(), b.p.cuda(), b.u.cuda(), i32(b.cu), draft_probs=own[1:])
    want, counts = b.want()
    assert (out.cpu().numpy() == want).all() and num.tolist() == counts
