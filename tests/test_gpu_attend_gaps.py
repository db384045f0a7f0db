"""The attention behind long stretches of prefix groups without keys: they are passed many at a time."""

import numpy as np
import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import latent as L
from test_gpu_latent import _bf, _cache, _good_rows

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


def _groups(T, prefixes, seed=5, block=16):
    """T tokens of one head, token t alone in group t, group t with prefixes.get(t, 0) keys, all from the same pages."""
    g = torch.Generator().manual_seed(seed)
    rows = _good_rows(g, 8 * block, R.BF16)
    val = R.values(rows, R.BF16)
    q = _bf(g, T, 1, 576)
    lens = torch.zeros(T, dtype=torch.int32)
    for t, n in prefixes.items():
        lens[t] = n
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None].expand(T, 8)
    offsets = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    qd, cache, ld = q.cuda(), _cache(rows, R.BF16, block), lens.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(**kw):
        return L.mla_prefix_decode_attention(qd, cache, kw.get("table"), kw.get("lens"), sm_scale=0.07, prefix_table=table,
                                             prefix_lens=ld, group_offsets=offsets, status=status)

    def check(out, lse):
        assert int(status.item()) == 0
        for t, n in prefixes.items():
            o, s, tol, stol = R.attend(q[t].double().numpy(), val[:n], 0.07)
            assert (np.abs(out[t].double().cpu().numpy() - o) <= tol).all(), t
            assert (np.abs(lse[t].double().cpu().numpy() - s) <= stol).all(), t
        rest = torch.ones(T, dtype=torch.bool, device="cuda")
        rest[list(prefixes)] = False
        assert (out[rest] == 0).all() and (lse[rest] == float("-inf")).all()
    return call, check


@pytest.mark.parametrize("gap", [1, 30, 31, 32, 33, 64, 100])
def test_attend_across_groups_without_keys(gap):
    prefixes = {gap * i + i: 1 + (13 * i) % 128 for i in range(40)}
    call, check = _groups(max(prefixes) + 1 + gap, prefixes)
    check(*call())


def test_attend_behind_groups_without_tokens():
    """Offsets padded with the number of tokens, lengths that belong to no one: passed on the way to the tokens."""
    T, block = 70, 16
    g = torch.Generator().manual_seed(8)
    rows = _good_rows(g, 8 * block, R.BF16)
    val = R.values(rows, R.BF16)
    q = _bf(g, T, 2, 576)
    offsets = torch.tensor([0, 20, 20, 25] + [T] * 67, dtype=torch.int32, device="cuda")
    lens = torch.tensor([40, 99, 0] + [128] * 67, dtype=torch.int32, device="cuda")
    own = torch.arange(T, dtype=torch.int32, device="cuda") % 30
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None].expand(T, 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = L.mla_prefix_decode_attention(q.cuda(), _cache(rows, R.BF16, block), table, own, sm_scale=0.07, prefix_table=table,
                                             prefix_lens=lens, group_offsets=offsets, status=status)
    assert int(status.item()) == 0
    for t in range(T):
        prefix = 40 if t < 20 else 0 if t < 25 else 128
        keys = np.concatenate([val[:prefix], val[:t % 30]])
        o, s, tol, stol = R.attend(q[t].double().numpy(), keys, 0.07)
        assert (np.abs(out[t].double().cpu().numpy() - o) <= tol).all(), t
        assert np.array_equal(lse[t].cpu().numpy(), s) if not len(keys) else (np.abs(lse[t].double().cpu().numpy() - s) <= stol).all(), t


def test_attend_passes_many_groups_without_keys_quickly():
    T = 100_000
    call, check = _groups(T, {0: 5, 1: 64, 50_000: 128, 50_001: 1, T - 2: 70})
    check(*call())
    # beside as many tokens without groups, which are passed 32 at a time
    q = torch.zeros((T, 1, 576), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((1, 16, 576), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda").expand(T, 1)
    lens = torch.zeros(T, dtype=torch.int32, device="cuda")
    lens[[0, T - 2]] = 5
    bare = _best_ms(lambda: L.mla_prefix_decode_attention(q, cache, table, lens, sm_scale=0.07))
    assert _best_ms(call) < 4 * bare + 0.2
