"""Weights that meet codes (k3da_chunk_attn over an e4m3 cache, few rows a kv
head), where what one key loses is too little to see and what all of them lose
is not, and where V's scales are next to the smallest (GPU).

Tolerance, from the arithmetic.  A weight is half precision, of a reference r
that stands 2^15 below the top of the range: off by 2^-12 of itself, or where
that is more (half's subnormal numbers, steps of 2^-24) by 2^-25 / 2^15 =
2^-40 of r, and r is at most 2^10 above the largest weight.  n keys that all
err one way are off by n * 2^-30 of the largest weight in sum: 2^-14 at 60000.
With values that are all v the output is then off by 2^-12 |v| (the weights),
2^-14 |v| (the small ones), less than 2^-10 |v| for the fp32 rest (sums of
60000 terms by 64 keys a product, ex2 within 2^-22) and 2^-8 |v| for its
rounding to bf16."""
import pytest
import torch

import speculative_decoding_drafter_k3_gb300 as k3da
from cache_cases import Batch, D, attend
from test_chunk_attn import call, dev

pytestmark = pytest.mark.gpu

ONE, MINUS_ONE, MINUS_EIGHT = 0x38, 0xB8, 0xD0  # e4m3 codes
UNIT = 127                                      # scale byte of 2^0


def leaders_and_a_tail(keys, spread, late):
    """One cache, for every request: scores of 0 for a leader in each of the
    first pages, 15.3 log2 units less for all other keys (q = 85 in dim 0:
    85 / 8 * log2 e), 122 less for one key next to each leader (`late`: 500
    pages further on) whose V row is 2^spread larger; values of 1."""
    b = Batch([1], [keys - 1], 24, 4, "e4m3", seed=1)
    code, byte = b.pool.view(torch.uint8), b.scales.view(torch.uint8)
    code[:, 0] = 0
    code[:, 0, :, :, 0] = MINUS_ONE
    code[:, 1] = ONE
    byte[:] = UNIT
    for j in range(16):
        at = int(b.table[0, j])
        code[at, 0, :, 0, 0] = 0
        far = int(b.table[0, j + (500 if late else 0)])
        code[far, 0, :, 1, 0] = MINUS_EIGHT
        byte[far, 1, :, 1] = UNIT + spread
    return b


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("spread", [0, 8, 10, 14])
def test_a_long_tail_of_small_weights_is_not_lost(spread, late):
    R, keys = 64, 60000
    b = leaders_and_a_tail(keys, spread, late)
    pool, scales, _, table, _, _ = dev(b)
    q = torch.zeros(R, 24, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 85.0
    q = q.view(R, 24 * D)
    out, lse = torch.empty_like(q), torch.empty(R, 24, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k3da.k3da_chunk_attn(out, q, pool, table.expand(R, -1).contiguous(),
                         torch.full((R,), keys - 1, dtype=torch.int32, device="cuda"),
                         torch.arange(R + 1, dtype=torch.int32, device="cuda"), num_q_heads=24, num_kv_heads=4,
                         kv_scales=scales, lse=lse, status=status,
                         workspace=k3da.alloc_chunk_workspace(R, R, 24, 4, b.stride))
    assert int(status) == 0
    x = torch.full((keys,), -85 / 8.0, dtype=torch.float64)
    x[torch.arange(16) * 64] = 0
    x[(torch.arange(16) + (500 if late else 0)) * 64 + 1] = -85.0
    # What the outlying rows bring is below 2^-100; all others are 1.
    err = (out.double() - 1).abs().max().item()
    assert err <= 2.0 ** -8 + 2.0 ** -12 + 2.0 ** -14 + 2.0 ** -10, f"off by {err:.4f}"
    want = torch.logsumexp(x, -1).item()
    assert (lse.double() - want).abs().max().item() <= 2.0 ** -24 * keys + 2.0 ** -20


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
