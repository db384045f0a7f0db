"""The gather over long stretches of sequences without rows: they are passed by search, not one load after another."""

import numpy as np
import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import latent as L
from test_gpu_latent import FMTS, NAMES, _cache, _good_rows, _kv_scale

pytestmark = pytest.mark.gpu


def _best_ms(f, n=5):
    f()
    times = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


def _gather(fmt, lens, block=4):
    g = torch.Generator().manual_seed(fmt)
    B, n = len(lens), int(sum(lens))
    rows = _good_rows(g, n, fmt)
    raw = np.full(((n + 2) * block, R.ROW_BYTES[fmt]), 0xFF, dtype=np.uint8)
    table = np.zeros((B, max(1, -(-max(lens) // block))), dtype=np.int32)
    at = page = 0
    for b in np.flatnonzero(lens):
        for k in range(lens[b]):
            if k % block == 0:
                table[b, k // block] = page
                page += 1
            raw[table[b, k // block] * block + k % block] = rows[at]
            at += 1
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
    cache, table = _cache(raw, fmt, block), torch.from_numpy(table).cuda()
    out = torch.full((n, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    return rows, out, lambda: L.mla_latent_cache_gather(cache, table, cu, n, out=out, kv_scale=_kv_scale(fmt))


def _check_rows(rows, out, fmt):
    val = R.values(rows, fmt, 0.05).astype(np.float32)
    if fmt == R.E4M3:
        val = (R.LUT[rows].astype(np.float32) * np.float32(0.05)).astype(np.float32)
    assert np.array_equal(out.cpu().view(torch.int16).numpy().view(np.uint16), R.bf16_bits(val))


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("gap", [1, 6, 7, 8, 9, 31, 32, 33, 1000])
def test_gather_across_empty_sequences(gap, fmt):
    """Gaps before, between and behind sequences of one to nine rows, so that a warp's eight rows lie on both sides."""
    lens = np.array([0] * gap + sum([[1 + i % 9] + [0] * (gap if i % 3 else 1) for i in range(25)], []) + [3] + [0] * gap)
    rows, out, call = _gather(fmt, lens)
    call()
    _check_rows(rows, out, fmt)


def test_gather_passes_long_gaps_quickly():
    lens = np.zeros(300_000, dtype=np.int64)
    lens[[0, 1, 150_000, 150_001, 299_998]] = 3
    rows, out, call = _gather(R.BF16, lens)
    call()
    _check_rows(rows, out, R.BF16)
    assert _best_ms(call) < 1.0  # 0.01 ms; with a load for each empty sequence 37
