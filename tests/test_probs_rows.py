"""Probabilities within a row (GPU): what is equal stays equal."""
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
