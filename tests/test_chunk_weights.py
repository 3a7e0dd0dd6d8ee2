"""V's scales next to the smallest, over an e4m3 cache (k3da_chunk_attn, GPU)."""
import pytest
import torch

from cache_cases import Batch, D, attend
from test_chunk_attn import call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("byte", [0, 1, 10, 40])
@pytest.mark.parametrize("new,ctx", [([1, 1], [900, 70]), ([1], [20000]), ([60], [900])])
def test_values_of_the_smallest_scales(new, ctx, byte):
    """V rows of code * 2^(byte - 127), code 256 to 448: normal bf16 numbers,
    2^-119 and up.  The tolerance of the definition (test_chunk_attn.py), by
    the power of two."""
    b = Batch(new, ctx, 6, 1, "e4m3", seed=2 + byte, stride=1300)
    code = b.pool.view(torch.uint8)
    g = torch.Generator().manual_seed(byte)
    code[:, 1] = torch.randint(0x78, 0x7F, code[:, 1].shape, generator=g, dtype=torch.uint8)
    b.scales.view(torch.uint8)[:, 1] = byte
    out, _ = call(b)
    want, _, mag, _ = attend(b, "causal")
    unit = 2.0 ** (byte - 127)
    got, want, mag = out.cpu().double().view(b.T, 6, D) / unit, want / unit, mag / unit
    err = (got - want).abs() - (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * mag)
    assert err.max() <= 0, f"off by {err.max():.3e} of the unit over its bound"
