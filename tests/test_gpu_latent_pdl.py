"""Insert, gather and attention as programmatic dependents of what comes before them on the stream: a producer that
writes their rows late, after it has let them start."""

import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import epilogue as E
from mla_decode_attention_10_b200 import latent as L
from mla_decode_attention_10_b200 import workloads as W
from test_gpu_latent import FMTS, NAMES, _bf, _cache, _kv_scale, SCALE

pytestmark = pytest.mark.gpu


def _bytes(cache):
    return cache.view(torch.uint8).reshape(-1, cache.shape[-1] * cache.element_size())


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("T", [1, 37, 1000])
def test_a_chain_of_dependents(T, fmt):
    """producer -> insert -> gather -> attention, each launched behind the one before, new rows every time."""
    g = torch.Generator().manual_seed(T)
    block, H = 16, 16
    pages = -(-T // block) + 1
    w = (1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16)
    tab = W.rope_table(T + 5)
    pos = torch.arange(T, dtype=torch.int32)
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    slots = perm[pos.long() // block].long() * block + pos.long() % block
    cache = _cache(torch.zeros((pages * block, R.ROW_BYTES[fmt]), dtype=torch.uint8).numpy(), fmt, block)
    wd, tabd, posd, slotd, table = w.cuda(), tab.cuda(), pos.cuda(), slots.cuda(), perm[None].cuda()
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    q = _bf(g, 1, H, 576).cuda()
    weights = torch.randint(0, 1 << 30, (16 << 20,), dtype=torch.int32, device="cuda")  # 64 MB, read before the rows are written
    sink = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv_c, k_pe = torch.zeros((T, 1, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, 1, 64), dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros((T, 576), dtype=torch.bfloat16, device="cuda")
    scale = _kv_scale(fmt)
    stream = torch.cuda.current_stream().cuda_stream
    want_bytes, got = [], []
    for i in range(4):
        src = _bf(g, T, 512), _bf(g, T, 64)
        want_bytes.append(R.insert_rows(*src, fmt, norm_weight=w, positions=pos, cos_sin=tab, kv_scale=SCALE))
        a, b = src[0].cuda(), src[1].cuda()
        torch.cuda.synchronize()
        rc = E.mla_harness_produce_after_weights(a.data_ptr(), b.data_ptr(), kv_c.data_ptr(), 512, 512, k_pe.data_ptr(), 64, 64,
                                                 weights.data_ptr(), 4 * weights.numel(), sink.data_ptr(), T, 1, 0, stream)
        assert rc == E.MLA_OK
        L.mla_latent_cache_insert(kv_c[:, 0], k_pe[:, 0], cache, slotd, norm_weight=wd, positions=posd, cos_sin=tabd,
                                  kv_scale=scale, pdl=True)
        L.mla_latent_cache_gather(cache, table, cu, T, out=rows, kv_scale=scale, pdl=True)
        out, lse = L.mla_prefix_decode_attention(q, cache, table, lens, sm_scale=0.07, kv_scale=scale, pdl=True)
        got.append((rows.clone(), out, lse, _bytes(cache)[slotd].cpu()))
    torch.cuda.synchronize()
    for want, (r, out, lse, raw) in zip(want_bytes, got):
        assert (raw.numpy() == want).all()
        val = R.values(want, fmt, SCALE)
        assert (abs(r.double().cpu().numpy() - val) <= abs(val) * R.EPS_BF16 + 1e-30).all()
        o, s, tol, stol = R.attend(q[0].double().cpu().numpy(), val, 0.07)
        assert (abs(out[0].double().cpu().numpy() - o) <= tol).all() and (abs(lse[0].double().cpu().numpy() - s) <= stol).all()
