"""One key far above a very long tail of keys, with e4m3 q and cache: the tail's weights are small, what they come to
together is not, and the sum has to have it as the denominator does.
"""

import math

import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import epilogue as E
from mla_decode_attention_10_b200 import latent as L

pytestmark = pytest.mark.gpu

FLOOR = 2.0 ** -29  # the contract's: a weight's absolute error, in weights of the row's largest


@pytest.mark.parametrize("x", [16, 20, 24, 26, 28])
def test_a_long_tail_of_small_weights(x):
    """Key 0 has score x ln 2 and no latents, the 2^18 - 1 others score 0 and latents 1: weights 1 and 2^-x.

    One token for every SM, so that each has its tail with its first key.  A weight is off by EPS_F8_WEIGHT and by
    FLOOR; the products' fp32 sum takes three terms of 32 keys at a time, each addition off by at most 2^-23 of it; the
    denominator adds a tile's weights at a time; ex2 and the scale add 2^-20; the result is rounded to bf16.
    """
    block, n = 64, 1 << 18
    T = torch.cuda.get_device_properties(0).multi_processor_count
    rows = torch.zeros((2 * block, 576), dtype=torch.uint8)
    one = R.e4m3_bytes(torch.ones(1).double().numpy())[0]
    rows[1:, :512] = int(one)
    rows[0, 512] = int(R.e4m3_bytes(torch.full((1,), float(x)).double().numpy())[0])
    cache = rows.view(2, block, 576).cuda()
    q = torch.zeros((T, 1, 576), dtype=torch.uint8, device="cuda")
    q[:, :, 512] = int(one)
    table = torch.ones((1, n // block), dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    unit = torch.ones(1, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = L.mla_prefix_decode_attention(
        q, cache, table.expand(T, -1), torch.full((T,), n, dtype=torch.int32, device="cuda"), sm_scale=math.log(2.0),
        q_scale=unit, kv_scale=unit, status=status)
    assert int(status.item()) == 0
    tail = (n - 1) * 2.0 ** -x
    want = tail / (1 + tail)
    adds = 3 * n / 32
    tol = want * (R.EPS_F8_WEIGHT + adds * 2.0 ** -23 + R.EPS_BF16 + 2.0 ** -20 + 2 * (n / 64) * 2.0 ** -23) + (n - 1) * FLOOR / (1 + tail)
    assert (out.double() - want).abs().max().item() <= tol
    ref = x * math.log(2.0) + math.log1p(tail)
    assert (lse.double() - ref).abs().max().item() <= 2.0 ** -20 + 2 * (n / 64) * 2.0 ** -23 + abs(ref) * 2.0 ** -21


def test_the_denominator_of_one_key_alone():
    """A row with a single key is that key, whatever its score: reference, lift and denominator cancel."""
    for code in (1.0, 448.0, -448.0):
        rows = torch.full((64, 576), int(R.e4m3_bytes(torch.full((1,), code).double().numpy())[0]), dtype=torch.uint8)
        q = torch.full((1, 16, 576), int(R.e4m3_bytes(torch.full((1,), 448.0).double().numpy())[0]), dtype=torch.uint8)
        unit = torch.ones(1, device="cuda")
        out, lse = L.mla_prefix_decode_attention(
            q.cuda(), rows.view(1, 64, 576).cuda(), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
            torch.ones(1, dtype=torch.int32, device="cuda"), sm_scale=1.0, q_scale=unit, kv_scale=unit)
        assert (out == code).all()
        s = 448.0 * code * 576  # fp32 holds it; log2 e and ln 2 each round it once more
        assert ((lse.double() - s).abs() <= abs(s) * 2.0 ** -21 + 2.0 ** -20).all()
