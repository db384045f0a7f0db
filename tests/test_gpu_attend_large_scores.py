"""Scores far beyond 2^24, where they are further apart than the softmax's own scale: a row is its largest key (or the
mean of several that tie), never zero; beyond 2^30 (2^27 with q and cache in e4m3) it may be NaN, all of it.

Scores are exact by construction: a query has one rotary value, 1, and key k's rotary value is a small integer.
"""

import numpy as np
import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import latent as L
from test_gpu_latent import KIND_IDS, KINDS, _cache

pytestmark = pytest.mark.gpu


def _raw(fmt, latents, rotary):
    kv, pe = torch.from_numpy(latents).to(torch.bfloat16), torch.zeros((len(rotary), 64), dtype=torch.bfloat16)
    pe[:, 0] = torch.from_numpy(rotary).to(torch.bfloat16)
    return R.insert_rows(kv, pe, fmt, kv_scale=1.0)


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [12, 20, 26, 30, 40, 60])
def test_large_scores(power, sign, fmt, q8):
    g = np.random.default_rng(power)
    block, H = 64, 16
    orders = [np.array([2.0]), np.arange(14.0) + 1, np.arange(14.0)[::-1] + 1, g.permutation(np.arange(300.0) % 13 + 1),
              np.sort(np.arange(4000.0) % 14 + 1), np.array([3.0, 1.0, 3.0, 2.0])]
    if sign < 0:
        orders = [o - 16.0 for o in orders]
    latents = [g.integers(-7, 8, (len(o), 512)).astype(np.float64) for o in orders]
    pages = [-(-len(o) // block) for o in orders]
    table = np.zeros((len(orders), max(pages)), dtype=np.int32)
    raw = np.full((sum(pages) * block, R.ROW_BYTES[fmt]), 0xFF, dtype=np.uint8)
    at = 0
    for t, (o, v) in enumerate(zip(orders, latents)):
        table[t, :pages[t]] = at + np.arange(pages[t])
        raw[at * block:at * block + len(o)] = _raw(fmt, v, o)
        at += pages[t]
    q = torch.zeros((len(orders), H, 576), dtype=torch.bfloat16)
    q[:, :, 512] = 1.0
    unit = torch.ones(1, device="cuda")
    if q8:
        q = torch.from_numpy(R.e4m3_bytes(q.double().numpy()))
    out, lse = L.mla_prefix_decode_attention(
        q.cuda(), _cache(raw, fmt, block), torch.from_numpy(table).cuda(),
        torch.tensor([len(o) for o in orders], dtype=torch.int32, device="cuda"), sm_scale=2.0 ** power,
        q_scale=unit if q8 else None, kv_scale=unit if fmt == R.E4M3 else None)
    for t, (o, v) in enumerate(zip(orders, latents)):
        most = 2.0 ** 27 if fmt == R.E4M3 and q8 else 2.0 ** 30
        if abs(o.max()) * 2.0 ** power >= most and torch.isnan(lse[t]).any():
            assert torch.isnan(lse[t]).all() and torch.isnan(out[t]).all()
            continue
        top = o == o.max()  # the others' weights are exp(-2^power) or less: zero
        want = v[top].mean(0)
        # equal weights, each rounded the same way; sums of integers are exact; one division and the result's rounding
        w = R.EPS_F8_WEIGHT if fmt == R.E4M3 and q8 else R.EPS_BF16
        assert (np.abs(out[t].double().cpu().numpy() - want) <= (w + 2.0 ** -20) * np.abs(v[top]).mean(0) + R.EPS_BF16 * np.abs(want)).all(), t
        s = o.max() * 2.0 ** power + np.log(top.sum())
        assert (np.abs(lse[t].double().cpu().numpy() - s) <= abs(s) * 2.0 ** -21).all(), t


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("power", [20, 30, 40, 60])
def test_scores_of_zero_among_very_low_ones(power, fmt, q8):
    """Keys far below -2^31 before, behind and around keys with a score of zero, in other tiles and other segments."""
    low, zero = lambda n: np.full(n, -5.0), lambda n: np.zeros(n)
    orders = [np.concatenate(p) for p in ((low(100), zero(3)), (zero(3), low(100)), (low(700), zero(1), low(700)),
                                          (low(4000), zero(5)), (low(30), zero(1), low(30)))]
    g = np.random.default_rng(power)
    block, H = 64, 16
    latents = [g.integers(-7, 8, (len(o), 512)).astype(np.float64) for o in orders]
    pages = [-(-len(o) // block) for o in orders]
    table = np.zeros((len(orders), max(pages)), dtype=np.int32)
    raw = np.full((sum(pages) * block, R.ROW_BYTES[fmt]), 0xFF, dtype=np.uint8)
    at = 0
    for t, (o, v) in enumerate(zip(orders, latents)):
        table[t, :pages[t]] = at + np.arange(pages[t])
        raw[at * block:at * block + len(o)] = _raw(fmt, v, o)
        at += pages[t]
    q = torch.zeros((len(orders), H, 576), dtype=torch.bfloat16)
    q[:, :, 512] = 1.0
    unit = torch.ones(1, device="cuda")
    if q8:
        q = torch.from_numpy(R.e4m3_bytes(q.double().numpy()))
    out, lse = L.mla_prefix_decode_attention(
        q.cuda(), _cache(raw, fmt, block), torch.from_numpy(table).cuda(),
        torch.tensor([len(o) for o in orders], dtype=torch.int32, device="cuda"), sm_scale=2.0 ** power,
        q_scale=unit if q8 else None, kv_scale=unit if fmt == R.E4M3 else None)
    for t, (o, v) in enumerate(zip(orders, latents)):
        want = v[o == 0].mean(0)
        w = R.EPS_F8_WEIGHT if fmt == R.E4M3 and q8 else R.EPS_BF16
        assert (np.abs(out[t].double().cpu().numpy() - want) <= (w + 2.0 ** -20) * np.abs(v[o == 0]).mean(0) + R.EPS_BF16 * np.abs(want)).all(), t
        assert (np.abs(lse[t].double().cpu().numpy() - np.log((o == 0).sum())) <= 2.0 ** -20).all(), t
