"""Attention where its rarer steps run: a maximum that moves within a segment, tile after tile, by more and by less than
the reference may lag; segments long enough for every lift of the e4m3 weights; infinities in q and in the cache."""

import numpy as np
import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import latent as L
from test_gpu_latent import KIND_IDS, KINDS, SCALE, _cache, _Case, _kv_scale

pytestmark = pytest.mark.gpu


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _queries(q, q8):
    """q fp64 [T, H, 576] as the kernel gets it, its scale, and the values it stands for."""
    if q8:
        raw = R.e4m3_bytes((q.astype(np.float32) / np.float32(SCALE)).astype(np.float64))
        return torch.from_numpy(raw).cuda(), torch.full((1,), SCALE, device="cuda"), R.LUT[raw] * float(np.float32(SCALE))
    t = torch.from_numpy(q).to(torch.bfloat16)
    return t.cuda(), None, t.double().numpy()


def _rows(x, fmt):
    t = torch.from_numpy(x).to(torch.bfloat16)
    raw = R.insert_rows(t[:, :512], t[:, 512:], fmt, kv_scale=SCALE)
    return raw, R.values(raw, fmt, SCALE)


def _rising(n_tiles, step, order):
    """Rotary value of each tile's keys: score `step` bits apart from tile to tile (q's is 4, the scale 1)."""
    i = {"up": np.arange(n_tiles), "down": np.arange(n_tiles)[::-1], "saw": np.arange(n_tiles) * 5 % n_tiles}[order]
    return np.repeat(i * step * np.log(2.0) / 4.0, 64)


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("order", ["up", "down", "saw"])
@pytest.mark.parametrize("step", [1.5, 7.0, 8.5, 11.0])
def test_moving_maximum_within_a_segment(step, order, fmt, q8):
    """A token for every SM, eleven tiles each, so that one segment has them all; four heads a token."""
    g = np.random.default_rng(3)
    tiles, T, H, block = 11, _sms(), 4, 64
    n = 64 * tiles - 7
    x = g.standard_normal((n, 576))
    x[:, 512] = _rising(tiles, step, order)[:n]
    raw, keys = _rows(x, fmt)
    raw = np.concatenate([raw, np.full((64 * tiles - n, raw.shape[1]), 0xFF, np.uint8)])
    q = g.standard_normal((T, H, 576)) * 0.04
    q[:, :, 512] = 4.0
    qd, q_scale, q64 = _queries(q, q8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = L.mla_prefix_decode_attention(
        qd, _cache(raw, fmt, block), torch.arange(tiles, dtype=torch.int32, device="cuda")[None].expand(T, tiles),
        torch.full((T,), n, dtype=torch.int32, device="cuda"), sm_scale=1.0, q_scale=q_scale, kv_scale=_kv_scale(fmt),
        status=status)
    assert int(status.item()) == 0
    o, s, tol, stol = R.attend(q64.reshape(T * H, 576), keys, 1.0, fmt == R.E4M3 and q8)
    assert (np.abs(out.double().cpu().numpy().reshape(T * H, 512) - o) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy().reshape(T * H) - s) <= stol).all()


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("block", [64, 20])
def test_moving_maximum_along_a_prefix(block, fmt, q8):
    """The same along a prefix of many rows (decoded into tiles where that is done), and from prefix to own keys."""
    g = np.random.default_rng(4)
    T, H, tiles = 24, 64, 9
    n = 64 * tiles + 11
    x = g.standard_normal((n + 40, 576))
    x[:n, 512] = np.resize(_rising(tiles, 9.0, "up"), n)
    x[n:, 512] = 16.0
    raw, keys = _rows(x, fmt)
    pages, own = -(-n // block), -(-40 // block)
    full = np.full(((pages + own) * block, raw.shape[1]), 0xFF, np.uint8)
    full[:n], full[pages * block:pages * block + 40] = raw[:n], raw[n:]
    q = g.standard_normal((T, H, 576)) * 0.04
    q[:, :, 512] = 4.0
    qd, q_scale, q64 = _queries(q, q8)
    lens = [(7 * t) % 41 for t in range(T)]
    out, lse = L.mla_prefix_decode_attention(
        qd, _cache(full, fmt, block), (pages + torch.arange(own, dtype=torch.int32, device="cuda"))[None].expand(T, own),
        torch.tensor(lens, dtype=torch.int32, device="cuda"), sm_scale=1.0,
        prefix_table=torch.arange(pages, dtype=torch.int32, device="cuda")[None],
        prefix_lens=torch.tensor([n], dtype=torch.int32, device="cuda"), q_scale=q_scale, kv_scale=_kv_scale(fmt))
    for t in range(T):
        o, s, tol, stol = R.attend(q64[t], np.concatenate([keys[:n], keys[n:n + lens[t]]]), 1.0, fmt == R.E4M3 and q8)
        assert (np.abs(out[t].double().cpu().numpy() - o) <= tol).all(), t
        assert (np.abs(lse[t].double().cpu().numpy() - s) <= stol).all(), t


@pytest.mark.parametrize("fmt,q8", [(R.E4M3, True), (R.BF16, False)], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("n", [8192, 8193, 20000, 70000])
def test_long_segments(n, fmt, q8):
    """Segments of so many keys (the same pages over and over), whose maximum rises from page to page of a round."""
    g = np.random.default_rng(n)
    T, H, block, distinct = _sms(), 2, 64, 16
    x = g.standard_normal((distinct * block, 576))
    x[:, 512] = _rising(distinct, 2.5, "saw")
    raw, keys = _rows(x, fmt)
    order = np.resize(np.arange(distinct), -(-n // block))
    order[:len(order) * 2 // 3] = order[:len(order) * 2 // 3] % 8  # the highest come late
    q = np.repeat(g.standard_normal((1, H, 576)) * 0.04, T, axis=0)
    q[:, :, 512] = 4.0
    qd, q_scale, q64 = _queries(q, q8)
    out, lse = L.mla_prefix_decode_attention(
        qd, _cache(raw, fmt, block), torch.from_numpy(order.astype(np.int32)).cuda()[None].expand(T, -1),
        torch.full((T,), n, dtype=torch.int32, device="cuda"), sm_scale=1.0, q_scale=q_scale, kv_scale=_kv_scale(fmt))
    all_keys = np.concatenate([keys[i * block:(i + 1) * block] for i in order])[:n]
    o, s, tol, stol = R.attend(q64[0], all_keys, 1.0, q8)
    assert (np.abs(out.double().cpu().numpy() - o) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - s) <= stol).all()


def _plant(case, token, key, at, bits):
    """Puts bf16 bits `bits` at rotary or latent value `at` of a token's key, in rows that hold it as bf16."""
    raw = case.cache.view(torch.uint8).view(-1, R.ROW_BYTES[case.fmt])
    slot = int(case.table[token, key // case.block]) * case.block + key % case.block
    byte = 2 * at if case.fmt == R.BF16 else 528 + 2 * (at - 512)
    raw[slot, byte:byte + 2] = torch.tensor([bits & 0xFF, bits >> 8], dtype=torch.uint8)


INF, MINUS_INF = 0x7F80, 0xFF80


@pytest.mark.parametrize("fmt", [R.BF16, R.MX], ids=["bf16", "mx"])
def test_infinite_rotary_values(fmt):
    """A key whose score is minus infinity counts for nothing, one whose score is infinity makes the row NaN: by head,
    as the query's sign has it.  Other tokens see neither."""
    case = _Case(fmt, 16, [70, 200, 5], seed=80)
    want = [x.clone() for x in case.call()]
    q = case.q64[1, :, 520]
    assert (q > 0).any() and (q < 0).any()
    _plant(case, 1, 130, 520, INF)
    out, lse = case.call()
    up, down = torch.from_numpy(q > 0).cuda(), torch.from_numpy(q < 0).cuda()
    assert torch.isnan(out[1, up]).all() and torch.isnan(lse[1, up]).all()
    case.keys[1] = np.delete(case.keys[1], 130, axis=0)
    for h in np.flatnonzero(q < 0):
        o, s, tol, stol = R.attend(case.q64[1, h:h + 1], case.keys[1], case.sm_scale)
        assert (np.abs(out[1, h].double().cpu().numpy() - o) <= tol).all() and abs(lse[1, h].item() - s) <= stol
    assert down.any() and torch.equal(out[[0, 2]], want[0][[0, 2]]) and torch.equal(lse[[0, 2]], want[1][[0, 2]])


def test_infinite_latents():
    """A latent of infinity: NaN rows where its score is infinity; where it is minus infinity, zero times infinity in
    that one column."""
    case = _Case(R.BF16, 16, [70, 200, 5], seed=81)
    want = [x.clone() for x in case.call()]
    q = case.q64[1, :, 33]
    assert (q > 0).any() and (q < 0).any()
    _plant(case, 1, 64, 33, MINUS_INF)
    out, lse = case.call()
    case.keys[1] = np.delete(case.keys[1], 64, axis=0)
    rest = np.arange(512) != 33
    for h in range(16):
        if q[h] < 0:
            assert torch.isnan(out[1, h]).all() and torch.isnan(lse[1, h])
        else:
            o, s, tol, stol = R.attend(case.q64[1, h:h + 1], case.keys[1], case.sm_scale)
            got = out[1, h].double().cpu().numpy()
            assert np.isnan(got[33]) and (np.abs(got - o[0]) <= tol[0])[rest].all() and abs(lse[1, h].item() - s) <= stol
    assert torch.equal(out[[0, 2]], want[0][[0, 2]]) and torch.equal(lse[[0, 2]], want[1][[0, 2]])


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
def test_a_query_that_is_not_a_number(fmt, q8):
    """NaN or infinity in one head's query: that row alone."""
    case = _Case(fmt, 16, [70, 200, 5], prefixes=[100], q8=q8, seed=82)
    want = [x.clone() for x in case.call()]
    case.q = case.q.clone()
    for h, bad in ((3, float("nan")), (9, float("inf"))):
        case.q[1, h, 7] = 0x7F if q8 else bad
    out, lse = case.call()
    hit = torch.zeros((3, 16), dtype=torch.bool, device="cuda")
    hit[1, 3] = hit[1, 9] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
