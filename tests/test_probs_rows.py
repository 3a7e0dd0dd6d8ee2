"""Probabilities within a row (GPU): what is equal stays equal, and each is as
near to its definition as the header says, at any distance below the largest
logit and any temperature."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def probs_of(x, cu, t):
    out = torch.full(x.shape, -3.0, device="cuda")
    k3da.k3da_token_probs(out, x.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                          temperatures=torch.tensor(t, dtype=torch.float32, device="cuda"))
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V", [(40, 700), (320, 4099), (40, 32768), (6, 32768), (3, 131075), (1, 300007)])
def test_equal_logits_have_equal_probabilities(T, V, dtype):
    """Bit for bit, whichever thread, warp or CTA of the row's cluster (of 1 to
    8) holds them; the parts of a row have largest logits of their own."""
    g = torch.Generator().manual_seed(V)
    x = ((torch.randn(T, V, generator=g) * 40).round() / 16).to(DTYPES[dtype])
    out = probs_of(x, [0, T], [0.7])
    x, at = x.cuda().float().sort(-1)
    out = out.gather(-1, at)
    alike, same = x[:, 1:] == x[:, :-1], out[:, 1:] == out[:, :-1]
    assert alike.any() and same[alike].all(), (int((~same)[alike].sum()), int(alike.sum()))


def check_near(got, x, t):
    """x [T, 8] as given, t [T].  With E = (x - top) / t a weight exp(E) is off by
    less than (n |E| + 9) 2^-24 of itself: half a step of each rounding in front
    of the power of two counts |E| 2^-24, the exponent's, the difference's where it
    is not exact, and with 16-bit logits that of 1 / t; the power of two's 2^-22
    counts twice, and its square is rounded.  The sum's terms bring theirs along,
    and up to 6 additions; 1 / sum and the product are rounded too."""
    short, top = x.dtype != torch.float32, x.float().amax(-1, keepdim=True)
    n = 1 + int(short) + (x.double() - top.double() != (x.float() - top).double()).numpy()
    x, t = x.double().numpy(), np.array(t, np.float32).astype(np.float64)[:, None]
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(x == -math.inf, -math.inf, (x - x.max(-1, keepdims=True)) / t)
    w = np.exp(e)
    off = np.where(e < 0, n * np.abs(np.where(w > 0, e, 0)) + 9, 0)
    total = w.sum(-1, keepdims=True)
    rel = 2.0 ** -24 * (off + (w * off).sum(-1, keepdims=True) / total + 8)
    want = w / total
    got = got.double().cpu().numpy()
    err = np.abs(got - want) / np.maximum(want, 2.0 ** -126)  # below, steps no longer shrink
    bad = err > rel + 2.0 ** -20 * (want < 2.0 ** -126)
    assert not bad.any(), (int(bad.sum()), t[bad.any(-1)][:3].tolist(), x[bad][:3], (err / rel).max())


@pytest.mark.parametrize("dtype", DTYPES)
def test_far_below_the_largest_logit(dtype):
    """Distances of up to 87 temperatures, large ones next to small ones, at
    temperatures of which some are those where log2(e) / t is furthest from
    fp32."""
    g = torch.Generator().manual_seed(1)
    t = torch.exp(torch.rand(200000, generator=g) * math.log(8.0)) * 0.3
    slope = 1 / (math.log(2.0) * t.double())
    off = ((slope.float().double() - slope) / slope).abs()
    t = torch.cat([torch.tensor([0.71901906]), t[:511], t[off.topk(512).indices]])
    x = torch.empty(1024, 8)
    x[:, 0] = 8 * torch.rand(1024, generator=g) * (torch.rand(1024, generator=g) < 0.5) + 8e-3 * torch.rand(1024, generator=g)
    x[:, 1:] = x[:, :1] - 87 * t[:, None] * torch.rand(1024, 7, generator=g)
    x[0, 0], x[0, 1:] = 8, -26.25
    x = x.to(DTYPES[dtype])
    check_near(probs_of(x, list(range(1025)), t.tolist()), x, t.tolist())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logits_and_temperatures_over_the_whole_range(dtype):
    """Temperatures of 2^-126 to 2^120, logits of their size and of the type's."""
    most = torch.finfo(DTYPES[dtype]).max
    parts = torch.tensor([1.0, -1.0, 0.0, 0.5, -0.25, 1e-3, -0.75, -math.inf], dtype=torch.float64)
    rows, t = [], []
    for tau in (2.0 ** -126, 1.7e-38, 1e-37, 2.0 ** -100, 1e-20, 2e-8, 1e-7, 1e-6, 0.9, 2.0 ** 24, 1e20, 2.0 ** 64, 1.2e30, 2.0 ** 120):
        for size in (most / 2, 20 * tau, 7 * tau, tau, 1.0, 2.0 ** -124):
            rows.append(parts * min(size, most / 2))
            t.append(tau)
    x, cu = torch.stack(rows).to(torch.float32).to(DTYPES[dtype]), list(range(len(t) + 1))
    check_near(probs_of(x, cu, t), x, t)
    # Below 2^-126 a temperature counts as that.
    least = probs_of(x, cu, [2.0 ** -126] * len(t))
    for tau in (1e-38, 1e-42, 2.0 ** -149):
        assert torch.equal(probs_of(x, cu, [tau] * len(t)), least)
    # At an infinite one the words that are not masked share the row: the longest
    # difference, 2^128, counts 2^-20 times log(2), twice.
    out = probs_of(x, cu, [math.inf] * len(t))
    assert (out[:, 7] == 0).all() and ((out[:, :7] - 1 / 7).abs() < 2.0 ** -19 / 7).all()


def test_a_difference_beyond_fp32_counts_as_infinite():
    most = torch.finfo(torch.float32).max
    x = torch.tensor([[most, -most, -0.5 * most, 0.0, -math.inf]])
    out = probs_of(x, [0, 1], [1e38])[0].tolist()
    assert out[1] == out[2] == out[4] == 0 and abs(out[3] / out[0] - math.exp(-most / float(torch.tensor(1e38)))) < 1e-6
