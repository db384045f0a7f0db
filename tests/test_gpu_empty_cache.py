"""A cache without pages, whose tensor has no address: there is nothing to read, and the calls say what they say of pages
that do not exist.  The epilogue with such a cache and no slots writes query rows only."""

import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import epilogue as E
from mla_decode_attention_10_b200 import latent as L
from mla_decode_attention_10_b200 import workloads as W
from test_gpu_latent import FMTS, KIND_IDS, KINDS, NAMES, _kv_scale

pytestmark = pytest.mark.gpu


def _empty(fmt, block=16):
    if fmt == R.BF16:
        return torch.empty((0, block, 576), dtype=torch.bfloat16, device="cuda")
    return torch.empty((0, block, R.ROW_BYTES[fmt]), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_gather(fmt):
    out = torch.full((5, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    for cu, want in (([0, 0, 0], 0), ([0, 2, 4], E.MLA_STATUS_SLOT_RANGE)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        L.mla_latent_cache_gather(_empty(fmt), table, torch.tensor(cu, dtype=torch.int32, device="cuda"), 5, out=out,
                                  kv_scale=_kv_scale(fmt), status=status)
        assert int(status.item()) == want and (out == 3.0).all()


@pytest.mark.parametrize("block", [16, 64, 20])
@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("T,H", [(3, 16), (20, 32)])
def test_attend(T, H, fmt, q8, block):
    q = torch.zeros((T, H, 576), dtype=torch.uint8 if q8 else torch.bfloat16, device="cuda")
    table = torch.zeros((T, 8), dtype=torch.int32, device="cuda")
    for n, want in ((0, 0), (100, E.MLA_STATUS_SLOT_RANGE)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lens = torch.full((T,), n, dtype=torch.int32, device="cuda")
        out, lse = L.mla_prefix_decode_attention(
            q, _empty(fmt, block), table, lens, sm_scale=1.0, prefix_table=table[:1], prefix_lens=lens[:1], kv_scale=_kv_scale(fmt),
            q_scale=torch.ones(1, device="cuda") if q8 else None, status=status)
        assert int(status.item()) == want
        assert (out == 0).all() and (lse == float("-inf")).all()


def test_query_rows_alone():
    w = W.make("queries", 37, 4, W.FLAG_ROPE, seed=2, num_blocks=4, rope_rows=128, cache_fill="random").to("cuda")
    want = torch.empty((37, 4, 576), dtype=torch.bfloat16, device="cuda")
    assert E.launch_workload(w, want) == E.MLA_OK
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = E.fused_mla_decode_q_concat_kv_cache_insert(
        w.q_nope, w.q_pe, w.kv_c, w.k_pe, _empty(R.BF16), torch.full((37,), -1, dtype=torch.int64, device="cuda"),
        positions=w.positions, cos_sin=w.cos_sin, status=status)
    assert torch.equal(q.view(torch.int16), want.view(torch.int16)) and int(status.item()) == 0
