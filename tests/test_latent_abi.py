"""The latent-cache entry points without a GPU: host arguments are rejected
before any CUDA call, the torch forms reject wrong tensors, and the tests' own
64-bit definitions agree with torch's conversions."""

import ctypes

import numpy as np
import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import build as B
from mla_decode_attention_10_b200 import epilogue as E
from mla_decode_attention_10_b200 import latent as L

A = 1 << 20  # a well-aligned address that nothing touches


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return E.lib()


def _insert(**kw):
    a = dict(kv_c=A, kv_c_stride_t=512, k_pe=A, k_pe_stride_t=64, slot_mapping=A, norm_weight=A, eps=1e-6, positions=A,
             cos_sin=A, rope_rows=8, kv_scale=A, T=4, block_size=64, num_blocks=1, format=E.MLA_CACHE_MX,
             flags=E.MLA_FLAG_ROPE, cache=A, status=None, stream=None)
    a.update(kw)
    return E.mla_latent_insert_launch(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=E.MLA_FLAG_Q_FP8), E.MLA_ERR_UNSUPPORTED),
    (dict(flags=1 << 31), E.MLA_ERR_UNSUPPORTED),
    (dict(format=3), E.MLA_ERR_UNSUPPORTED),
    (dict(format=-1), E.MLA_ERR_UNSUPPORTED),
    (dict(T=-1), E.MLA_ERR_INVALID_ARG),
    (dict(T=2 ** 31), E.MLA_ERR_INVALID_ARG),
    (dict(block_size=0), E.MLA_ERR_INVALID_ARG),
    (dict(num_blocks=-1), E.MLA_ERR_INVALID_ARG),
    (dict(num_blocks=2 ** 50), E.MLA_ERR_INVALID_ARG),
    (dict(eps=-1e-6), E.MLA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), E.MLA_ERR_INVALID_ARG),
    (dict(eps=float("inf")), E.MLA_ERR_INVALID_ARG),
    (dict(kv_c=None), E.MLA_ERR_INVALID_ARG),
    (dict(k_pe=None), E.MLA_ERR_INVALID_ARG),
    (dict(slot_mapping=None), E.MLA_ERR_INVALID_ARG),
    (dict(cache=None), E.MLA_ERR_INVALID_ARG),
    (dict(positions=None), E.MLA_ERR_INVALID_ARG),
    (dict(cos_sin=None), E.MLA_ERR_INVALID_ARG),
    (dict(rope_rows=0), E.MLA_ERR_INVALID_ARG),
    (dict(format=E.MLA_CACHE_E4M3, kv_scale=None), E.MLA_ERR_INVALID_ARG),
    (dict(kv_c_stride_t=-8), E.MLA_ERR_INVALID_ARG),
    (dict(kv_c=A + 8), E.MLA_ERR_ALIGNMENT),
    (dict(kv_c_stride_t=516), E.MLA_ERR_ALIGNMENT),
    (dict(cache=A + 8), E.MLA_ERR_ALIGNMENT),
    (dict(norm_weight=A + 2), E.MLA_ERR_ALIGNMENT),
    (dict(k_pe=A + 1), E.MLA_ERR_ALIGNMENT),
    (dict(slot_mapping=A + 4), E.MLA_ERR_ALIGNMENT),
    (dict(positions=A + 2), E.MLA_ERR_ALIGNMENT),
    (dict(status=A + 1), E.MLA_ERR_ALIGNMENT),
    (dict(T=0, kv_c=None, k_pe=None, slot_mapping=None, cache=None), E.MLA_OK),
])
def test_insert_arguments(kw, code):
    assert _insert(**kw) == code


def _gather(**kw):
    a = dict(cache=A, format=E.MLA_CACHE_MX, block_size=64, num_blocks=4, kv_scale=A, block_table=A, table_stride=2,
             table_cols=2, cu_rows=A, first=A, B=2, N=10, flags=0, out=A, out_stride=576, status=None, stream=None)
    a.update(kw)
    return E.mla_latent_gather_launch(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=E.MLA_FLAG_ROPE), E.MLA_ERR_UNSUPPORTED),
    (dict(format=7), E.MLA_ERR_UNSUPPORTED),
    (dict(B=-1), E.MLA_ERR_INVALID_ARG),
    (dict(N=-1), E.MLA_ERR_INVALID_ARG),
    (dict(N=2 ** 31), E.MLA_ERR_INVALID_ARG),
    (dict(block_size=0), E.MLA_ERR_INVALID_ARG),
    (dict(table_cols=-1), E.MLA_ERR_INVALID_ARG),
    (dict(table_stride=-1), E.MLA_ERR_INVALID_ARG),
    (dict(cache=None), E.MLA_ERR_INVALID_ARG),
    (dict(block_table=None), E.MLA_ERR_INVALID_ARG),
    (dict(cu_rows=None), E.MLA_ERR_INVALID_ARG),
    (dict(out=None), E.MLA_ERR_INVALID_ARG),
    (dict(out_stride=575), E.MLA_ERR_INVALID_ARG),
    (dict(format=E.MLA_CACHE_E4M3, kv_scale=None), E.MLA_ERR_INVALID_ARG),
    (dict(out_stride=580), E.MLA_ERR_ALIGNMENT),
    (dict(out=A + 8), E.MLA_ERR_ALIGNMENT),
    (dict(cache=A + 8), E.MLA_ERR_ALIGNMENT),
    (dict(cu_rows=A + 2), E.MLA_ERR_ALIGNMENT),
    (dict(first=A + 2), E.MLA_ERR_ALIGNMENT),
    (dict(N=0, cache=None, out=None), E.MLA_OK),
    (dict(B=0, cache=None, cu_rows=None), E.MLA_OK),
])
def test_gather_arguments(kw, code):
    assert _gather(**kw) == code


def _attend(**kw):
    a = dict(q=A, q_stride_t=16 * 576, q_stride_h=576, q_scale=A, cache=A, format=E.MLA_CACHE_BF16, block_size=64,
             num_blocks=4, kv_scale=A, prefix_table=A, prefix_stride=2, prefix_cols=2, prefix_lens=A, group_offsets=A,
             G=1, block_table=A, table_stride=2, table_cols=2, seq_lens=A, T=4, H=16, sm_scale=0.07, flags=0, out=A,
             lse=A, workspace=A, workspace_bytes=1 << 40, status=None, stream=None)
    a.update(kw)
    return E.mla_prefix_attend_launch(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=E.MLA_FLAG_ROPE), E.MLA_ERR_UNSUPPORTED),
    (dict(format=3), E.MLA_ERR_UNSUPPORTED),
    (dict(T=-1), E.MLA_ERR_INVALID_ARG),
    (dict(H=0), E.MLA_ERR_INVALID_ARG),
    (dict(H=65536), E.MLA_ERR_INVALID_ARG),
    (dict(T=2 ** 27, H=16), E.MLA_ERR_INVALID_ARG),
    (dict(G=-1), E.MLA_ERR_INVALID_ARG),
    (dict(G=5), E.MLA_ERR_INVALID_ARG),
    (dict(block_size=0), E.MLA_ERR_INVALID_ARG),
    (dict(num_blocks=-1), E.MLA_ERR_INVALID_ARG),
    (dict(table_cols=-1), E.MLA_ERR_INVALID_ARG),
    (dict(prefix_cols=0), E.MLA_ERR_INVALID_ARG),
    (dict(sm_scale=float("nan")), E.MLA_ERR_INVALID_ARG),
    (dict(sm_scale=float("inf")), E.MLA_ERR_INVALID_ARG),
    (dict(q=None), E.MLA_ERR_INVALID_ARG),
    (dict(cache=None), E.MLA_ERR_INVALID_ARG),
    (dict(out=None), E.MLA_ERR_INVALID_ARG),
    (dict(workspace=None), E.MLA_ERR_INVALID_ARG),
    (dict(flags=E.MLA_FLAG_Q_FP8, q_scale=None), E.MLA_ERR_INVALID_ARG),
    (dict(format=E.MLA_CACHE_E4M3, kv_scale=None), E.MLA_ERR_INVALID_ARG),
    (dict(prefix_table=None), E.MLA_ERR_INVALID_ARG),
    (dict(prefix_lens=None), E.MLA_ERR_INVALID_ARG),
    (dict(G=2, group_offsets=None), E.MLA_ERR_INVALID_ARG),
    (dict(block_table=None), E.MLA_ERR_INVALID_ARG),
    (dict(seq_lens=None), E.MLA_ERR_INVALID_ARG),
    (dict(q_stride_t=-8), E.MLA_ERR_INVALID_ARG),
    (dict(q=A + 8), E.MLA_ERR_ALIGNMENT),
    (dict(out=A + 8), E.MLA_ERR_ALIGNMENT),
    (dict(cache=A + 8), E.MLA_ERR_ALIGNMENT),
    (dict(workspace=A + 128), E.MLA_ERR_ALIGNMENT),
    (dict(q_stride_h=580), E.MLA_ERR_ALIGNMENT),
    (dict(flags=E.MLA_FLAG_Q_FP8, q_stride_h=584), E.MLA_ERR_ALIGNMENT),
    (dict(lse=A + 2), E.MLA_ERR_ALIGNMENT),
    (dict(seq_lens=A + 2), E.MLA_ERR_ALIGNMENT),
    (dict(T=0, G=0, q=None, cache=None, out=None, workspace=None), E.MLA_OK),
])
def test_attend_arguments(kw, code):
    assert _attend(**kw) == code


def test_attend_workspace():
    w = E.mla_prefix_attend_workspace
    assert 0 < w(1, 16, 0, 0, 148) < w(64, 16, 0, 0, 148) < w(64, 16, 1, 0, 148) < w(64, 16, 1, 8192, 148)
    # a prefix of few rows is not decoded into the workspace, however long
    assert w(4, 16, 1, 8192, 148) == w(4, 16, 1, 1 << 40, 148)
    n = ctypes.c_int64()
    for args in ((-1, 16, 0, 0), (1, 0, 0, 0), (1, 16, 2, 0), (1, 16, -1, 0), (1, 16, 0, -1), (2 ** 30, 16, 0, 0)):
        assert E.lib().mla_prefix_attend_workspace(*args, 148, ctypes.byref(n)) == E.MLA_ERR_INVALID_ARG
    assert E.lib().mla_prefix_attend_workspace(1, 16, 0, 0, 148, None) == E.MLA_ERR_INVALID_ARG


def test_cuda_failures_are_recorded():
    if torch.cuda.is_available():
        pytest.skip("needs a process without a visible GPU")
    for call in (_insert, _gather, _attend, lambda: E.lib().mla_prefix_attend_workspace(
            4, 16, 0, 0, 0, ctypes.byref(ctypes.c_int64()))):
        assert call() == E.MLA_ERR_CUDA
        assert E.last_cuda_error() != 0


def test_torch_forms_reject_host_tensors():
    cache = torch.zeros((2, 16, 576), dtype=torch.bfloat16)
    x, pe, slots = torch.zeros((3, 512), dtype=torch.bfloat16), torch.zeros((3, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        L.mla_latent_cache_insert(x, pe, cache, slots)
    table, cu = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        L.mla_latent_cache_gather(cache, table, cu, 1)
    with pytest.raises(ValueError, match="CUDA"):
        L.mla_prefix_decode_attention(torch.zeros((1, 1, 576), dtype=torch.bfloat16), cache, table, cu[:1], sm_scale=1.0)


# ---- the tests' definitions ---------------------------------------------------------------

def test_reference_e4m3_agrees_with_torch():
    x = torch.cat([torch.arange(0, 65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float(),
                   torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 100])
    x = x[torch.isfinite(x)]
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_bytes(x.double().numpy()), want)
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    v = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(R.LUT)) and np.array_equal(v[~np.isnan(v)], R.LUT[~np.isnan(v)])


def test_reference_bf16_agrees_with_torch():
    x = torch.randn(50000, generator=torch.Generator().manual_seed(2)) * torch.logspace(-38, 38, 50000)
    assert np.array_equal(R.bf16_bits(x.numpy()).view(np.int16), x.to(torch.bfloat16).view(torch.int16).numpy())


def test_reference_microscaling_keeps_each_value_within_half_a_step():
    g = torch.Generator().manual_seed(3)
    x = torch.ldexp(torch.randn(40, 512, generator=g), torch.randint(-30, 30, (40, 512), generator=g)).to(torch.bfloat16)
    rows = R.insert_rows(x, torch.zeros(40, 64, dtype=torch.bfloat16), R.MX)
    v, x = R.values(rows, R.MX)[:, :512], x.double().numpy()
    e = rows[:, 512:528].astype(np.float64) - 127
    unit = np.repeat(2.0 ** e, 32, axis=1)
    a = np.abs(x) / unit
    assert a.max() <= 448
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    assert (np.abs(v - x) / unit <= step / 2).all()
    # and the exponent is the least: half of it would not hold the group's largest
    top = np.abs(x).reshape(40, 16, 32).max(-1)
    assert (top > 448 * 2.0 ** (e - 1)).all()


def test_reference_attention_agrees_with_torch():
    g = torch.Generator().manual_seed(4)
    q, k = torch.randn(3, 576, generator=g, dtype=torch.float64), torch.randn(50, 576, generator=g, dtype=torch.float64)
    out, lse, _, _ = R.attend(q.numpy(), k.numpy(), 0.07)
    s = q @ k.t() * 0.07
    assert np.allclose(out, (torch.softmax(s, -1) @ k[:, :512]).numpy(), atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(s, -1).numpy(), atol=1e-12)
