"""The attention kernel's way out when one of its bounded waits runs out: it returns, says so in the status, and rows
that a CTA which gave up had a part in are NaN, never what an earlier call left in the workspace.

The waits are made to run out by a small number of tries; nothing hangs and the context stays usable.
"""

import numpy as np
import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import epilogue as E
from test_gpu_latent import KIND_IDS, KINDS, _Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def restore():
    yield
    E.mla_harness_attend_spins()


def _workspace(case):
    cap = case.prefix_table.shape[1] * case.block if case.prefixes else 0
    n = E.mla_prefix_attend_workspace(len(case.lens), case.H, len(case.prefixes), cap)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def _call(case, ws):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = case.call(status=status, workspace=ws)
    return out, lse, int(status.item())


def _cases(fmt, q8):
    # own keys alone, some rows without any; a prefix for many rows (decoded into tiles where that is done)
    yield _Case(fmt, 16, [700, 0, 64, 3], q8=q8, seed=1)
    yield _Case(fmt, 32, [(13 * i) % 50 for i in range(40)], prefixes=[300, 129], members=[0, 17, 40], block=64, q8=q8, seed=2)


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
def test_hardly_any_patience(fmt, q8):
    for case in _cases(fmt, q8):
        ws = _workspace(case)
        out, lse, st = _call(case, ws)  # leaves its partial sums in the workspace
        assert st == 0
        case.check(out, lse)
        E.mla_harness_attend_spins(0)
        out, lse, st = _call(case, ws)
        assert st == E.MLA_STATUS_TIMEOUT
        some = torch.tensor([case.keys_of(t).shape[0] > 0 for t in range(len(case.lens))], device="cuda")
        assert torch.isnan(out[some]).all() and torch.isnan(lse[some]).all()
        assert (out[~some] == 0).all() and (lse[~some] == float("-inf")).all()
        E.mla_harness_attend_spins()
        out, lse, st = _call(case, ws)
        assert st == 0
        case.check(out, lse)


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
def test_little_patience(fmt, q8):
    """Whichever wait runs out, and wherever the others are by then: a row is right or NaN, and NaN only with the status."""
    for case in _cases(fmt, q8):
        ws = _workspace(case)
        right = _call(case, ws)[:2]
        case.check(*right)
        for spins in (1, 30, 50, 70, 100, 140, 200, 1000):
            E.mla_harness_attend_spins(spins)
            out, lse, st = _call(case, ws)
            assert st in (0, E.MLA_STATUS_TIMEOUT)
            nan = torch.isnan(lse)
            assert torch.equal(nan[..., None].expand_as(out), torch.isnan(out))
            assert st == E.MLA_STATUS_TIMEOUT or not nan.any()
            assert torch.equal(lse[~nan], right[1][~nan])
            assert torch.equal(out[~nan].view(torch.int16), right[0][~nan].view(torch.int16))
        E.mla_harness_attend_spins()
        out, lse, st = _call(case, ws)
        assert st == 0 and torch.equal(out.view(torch.int16), right[0].view(torch.int16)) and torch.equal(lse, right[1])


def test_a_captured_call_keeps_its_patience():
    """The number of tries is the call's own: a graph captured before a change replays as captured."""
    case = _Case(R.BF16, 16, [100, 30], prefixes=[80], seed=3)
    case.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = case.call()
    E.mla_harness_attend_spins(0)
    g.replay()
    torch.cuda.synchronize()
    case.check(out, lse)
    assert np.isfinite(lse.cpu().numpy()).all()
