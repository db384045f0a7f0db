"""The workspace of the attention over the latent cache: what a call of a given cache takes, and no more."""

import ctypes

import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import build as B
from mla_decode_attention_10_b200 import epilogue as E
from mla_decode_attention_10_b200 import latent as L

A = 1 << 20  # a well-aligned address that nothing touches
Q8 = E.MLA_FLAG_Q_FP8


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return E.lib()


SIZES = [(1, 16, 0, 0), (64, 16, 1, 131072), (64, 16, 4, 8192), (63, 4, 1, 8192), (1024, 16, 14, 131072), (4096, 128, 3, 64)]


@pytest.mark.parametrize("T,H,G,keys", SIZES)
def test_never_more_than_for_any_cache(T, H, G, keys):
    most = E.mla_prefix_attend_workspace(T, H, G, keys, 148)
    for fmt in (R.BF16, R.E4M3, R.MX):
        for flags in (0, Q8):
            for block, blocks in ((64, 100), (20, 100), (1, 10), (64, 0), (64, 2 ** 26), (64, 2 ** 40)):
                assert 0 < E.mla_prefix_attend_workspace_for(T, H, G, keys, fmt, flags, block, blocks, 148) <= most


def test_images_only_where_a_call_makes_them():
    def need(fmt, flags, block, blocks=1000, keys=131072, T=64):
        return E.mla_prefix_attend_workspace_for(T, 16, 1, keys, fmt, flags, block, blocks, 148)
    bare, most = E.mla_prefix_attend_workspace(64, 16, 1, 0, 148), E.mla_prefix_attend_workspace(64, 16, 1, 131072, 148)
    assert most - bare == 131072 // 64 * 73856
    # whole tiles by tensor copies: no images
    for fmt, flags in ((R.BF16, 0), (R.BF16, Q8), (R.E4M3, Q8)):
        for block in (8, 16, 64, 100 * 64):
            assert need(fmt, flags, block) == bare
    # rows to be decoded, odd pages, more rows than a tensor copy can number, a cache without pages
    for fmt, flags, block, blocks in ((R.MX, 0, 64, 1000), (R.MX, Q8, 64, 1000), (R.E4M3, 0, 64, 1000), (R.BF16, 0, 20, 1000),
                                      (R.BF16, 0, 64, 2 ** 25), (R.BF16, 0, 64, 0)):
        assert need(fmt, flags, block, blocks) == most
    codes = need(R.E4M3, Q8, 20)  # images of codes are smaller
    assert codes - bare == 131072 // 64 * (5 * 8192 + 128)
    # few rows: none for any cache
    assert need(R.MX, 0, 64, T=15) == E.mla_prefix_attend_workspace(15, 16, 1, 0, 148)


def test_arguments():
    n = ctypes.c_int64()
    good = dict(T=4, H=16, G=1, prefix_keys=64, format=R.MX, flags=0, block_size=64, num_blocks=4, sm_count=148)

    def call(bytes=ctypes.byref(n), **kw):
        return E.lib().mla_prefix_attend_workspace_for(*{**good, **kw}.values(), bytes)
    assert call() == E.MLA_OK and n.value > 0
    for kw in (dict(format=3), dict(format=-1), dict(flags=E.MLA_FLAG_ROPE)):
        assert call(**kw) == E.MLA_ERR_UNSUPPORTED
    for kw in (dict(T=-1), dict(H=0), dict(G=5), dict(prefix_keys=-1), dict(block_size=0), dict(num_blocks=-1),
               dict(num_blocks=2 ** 50), dict(bytes=None)):
        assert call(**kw) == E.MLA_ERR_INVALID_ARG


def _launch(need, **kw):
    a = dict(q=A, q_stride_t=16 * 576, q_stride_h=576, q_scale=A, cache=A, format=R.BF16, block_size=64, num_blocks=1000,
             kv_scale=A, prefix_table=A, prefix_stride=2048, prefix_cols=2048, prefix_lens=A, group_offsets=A, G=1,
             block_table=A, table_stride=2, table_cols=2, seq_lens=A, T=64, H=16, sm_scale=0.07, flags=0, out=A, lse=A,
             workspace=A, workspace_bytes=need, status=None, stream=None)
    a.update(kw)
    return E.mla_prefix_attend_launch(**a)


@pytest.mark.gpu
def test_a_byte_too_few_is_refused():
    for fmt in (R.BF16, R.MX):
        need = E.mla_prefix_attend_workspace_for(64, 16, 1, 131072, fmt, 0, 64, 1000)
        assert _launch(need - 1, format=fmt) == E.MLA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,q8", [(f, q) for f in (R.BF16, R.E4M3, R.MX) for q in (False, True)])
@pytest.mark.parametrize("block", [64, 20])
def test_a_call_keeps_to_its_workspace(block, fmt, q8):
    from test_gpu_latent import _Case
    case = _Case(fmt, 32, [(13 * i) % 50 for i in range(40)], prefixes=[300, 129], members=[0, 17, 40], block=block, q8=q8,
                 seed=block, pad_cols=50)
    need = E.mla_prefix_attend_workspace_for(40, 32, 2, case.prefix_table.shape[1] * block, fmt, Q8 if q8 else 0, block,
                                             case.cache.shape[0])
    guard = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = case.call(status=status, workspace=guard[:need])
    case.check(out, lse)
    assert int(status.item()) == 0 and (guard[need:] == 0x5A).all()


@pytest.mark.gpu
def test_the_torch_form_takes_what_the_cache_needs():
    """A wide table of a cache that is copied as it is: no room for images that nothing writes."""
    T, H, block, cols = 64, 16, 64, 2048
    cache = torch.zeros((4, block, 576), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((T, H, 576), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, cols), dtype=torch.int32, device="cuda")
    lens = torch.full((1,), 100, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out, lse = L.mla_prefix_decode_attention(q, cache, None, None, sm_scale=1.0, prefix_table=table, prefix_lens=lens)
    assert (out == 0).all()
    taken = torch.cuda.max_memory_allocated() - before
    assert taken < E.mla_prefix_attend_workspace(T, H, 1, 0) + 4 * out.numel() + 2 ** 20
