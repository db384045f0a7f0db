"""Latent cache rows written with norm, rotation and quantisation, read back,
and attended to with shared prefixes, against plain 64-bit definitions.

Insert and gather are compared bit for bit: the norm is held in 64 bits and
rounded once, every other step is exact or has one defined rounding.  The
attention's tolerances are derived in ``latent_ref.attend``.

Cache rows that no sequence owns, and rows behind a sequence's end in its last
page, hold NaN throughout, so a read of one of them shows in the result.
"""

import numpy as np
import pytest
import torch

import latent_ref as R
from mla_decode_attention_10_b200 import epilogue as E
from mla_decode_attention_10_b200 import latent as L
from mla_decode_attention_10_b200 import workloads as W

pytestmark = pytest.mark.gpu

FMTS = [R.BF16, R.E4M3, R.MX]
NAMES = {R.BF16: "bf16", R.E4M3: "e4m3", R.MX: "mx"}
SCALE = 0.05


def _bf(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def _cache(raw: np.ndarray, fmt: int, block: int) -> torch.Tensor:
    t = torch.from_numpy(raw).cuda().view(-1, block, raw.shape[1])
    return t.view(torch.bfloat16) if fmt == R.BF16 else t


def _bytes(cache: torch.Tensor) -> np.ndarray:
    c = cache.contiguous().view(torch.uint8)
    return c.view(-1, c.shape[-1]).cpu().numpy()


def _kv_scale(fmt):
    return torch.full((1,), SCALE, device="cuda") if fmt == R.E4M3 else None


# ---- insert -----------------------------------------------------------------------------

def _insert_case(T, fmt, norm, rope, seed, std=1.0, row=512, block=16, spread=False):
    g = torch.Generator().manual_seed(seed)
    kv = _bf(g, T, row, std=std)
    if spread:  # magnitudes over the whole range of the type
        kv = torch.ldexp(kv.float(), torch.randint(-120, 120, (T, row), generator=g)).to(torch.bfloat16)
    kv = kv[:, row - 512:]
    pe = _bf(g, T, 70)[:, :64]
    w = (1 + 0.2 * torch.randn(512, generator=g)).to(torch.bfloat16) if norm else None
    n_blocks = T // block + 2
    slots = torch.randperm(n_blocks * block, generator=g)[:T]
    pos = torch.randint(0, 300, (T,), generator=g, dtype=torch.int32) if rope else None
    tab = W.rope_table(300) if rope else None
    raw = torch.randint(0, 256, (n_blocks * block, R.ROW_BYTES[fmt]), generator=g, dtype=torch.uint8).numpy()
    return kv, pe, w, slots, pos, tab, raw, block


def _move(t):
    return None if t is None else W._move(t, "cuda")


def _run_insert(case, fmt, **kw):
    kv, pe, w, slots, pos, tab, raw, block = case
    cache = _cache(raw, fmt, block)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.mla_latent_cache_insert(_move(kv), _move(pe), cache, _move(slots), norm_weight=_move(w),
                              positions=_move(pos), cos_sin=_move(tab), kv_scale=_kv_scale(fmt), status=status, **kw)
    torch.cuda.synchronize()
    want = raw.copy()
    ok = (slots >= 0) & (slots < raw.shape[0])
    rows = R.insert_rows(kv, pe, fmt, norm_weight=w, positions=pos, cos_sin=tab, kv_scale=SCALE)
    want[slots[ok].numpy()] = rows[ok.numpy()]
    return _bytes(cache), want, int(status.item())


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("norm,rope", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("T", [1, 2, 149, 700])
def test_insert_rows_bit_for_bit(T, norm, rope, fmt):
    got, want, st = _run_insert(_insert_case(T, fmt, norm, rope, seed=T + 7 * fmt), fmt)
    assert st == 0
    assert np.array_equal(got, want)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("norm", [False, True])
def test_insert_strided_latents_and_many_rows(norm, fmt):
    got, want, _ = _run_insert(_insert_case(3000, fmt, norm, True, seed=5, row=1536, std=3.0), fmt)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("norm", [False, True])
def test_insert_values_of_every_magnitude(norm, fmt):
    got, want, _ = _run_insert(_insert_case(64, fmt, norm, False, seed=9, spread=True), fmt)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_insert_special_values(fmt):
    """Zeros of both signs, subnormals, the largest numbers, infinities and NaN, without a norm."""
    case = list(_insert_case(6, fmt, False, False, seed=3))
    kv = torch.zeros(6, 512, dtype=torch.bfloat16)
    kv[0, 1::2] = -0.0
    kv[1] = 2.0 ** -130
    kv[2] = 3.38e38
    kv[2, 100:] = 1.0
    kv[3, :40] = float("inf")
    kv[3, 40:] = 2.0
    kv[4, ::7] = float("nan")
    kv[4, 1::7] = -float("inf")
    kv[4, 2::7] = 448.0
    kv[5] = torch.linspace(-448, 448, 512).to(torch.bfloat16)
    case[0] = kv
    got, want, _ = _run_insert(tuple(case), fmt)
    if fmt == R.BF16 or fmt == R.MX:
        assert np.array_equal(got, want)
    else:  # a NaN code may carry either sign
        same = (got == want) | ((got & 0x7F == 0x7F) & (want & 0x7F == 0x7F))
        assert same.all()


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_insert_skips_bad_slots_and_positions(fmt):
    case = list(_insert_case(40, fmt, True, True, seed=21))
    case[3][3] = -1
    case[3][7] = case[6].shape[0]
    case[3][9] = 2 ** 40
    case[4][11] = -1
    case[4][12] = 300
    got, want, st = _run_insert(tuple(case), fmt)
    assert st == E.MLA_STATUS_SLOT_RANGE | E.MLA_STATUS_POS_RANGE
    assert np.array_equal(got, want)


def test_insert_matches_the_epilogue_row():
    """Without a norm the row is the one mla_epilogue_launch writes, byte for byte."""
    for flags, fmt in ((W.FLAG_ROPE, R.BF16), (W.FLAG_ROPE | W.FLAG_KV_FP8, R.E4M3)):
        w = W.make("same", 37, 4, flags, seed=2, num_blocks=2, rope_rows=128, cache_fill="random").to("cuda")
        mine = w.cache.clone()
        q = torch.empty((37, 4, 576), dtype=torch.bfloat16, device="cuda")
        assert E.launch_workload(w, q) == E.MLA_OK
        L.mla_latent_cache_insert(w.kv_c, w.k_pe, mine, w.slot_mapping, positions=w.positions, cos_sin=w.cos_sin,
                                  kv_scale=w.kv_scale)
        assert torch.equal(mine.view(torch.uint8), w.cache.view(torch.uint8))


# ---- gather -----------------------------------------------------------------------------

def _good_rows(g, n, fmt):
    """Byte rows without NaN or infinity, codes and scale exponents over their whole range."""
    if fmt == R.BF16:
        x = torch.randn(n, 576, generator=g).to(torch.bfloat16)
        return x.view(torch.uint8).numpy().reshape(n, R.ROW_BYTES[fmt]).copy()
    codes = torch.randint(0, 126, (n, R.ROW_BYTES[fmt]), generator=g).to(torch.uint8)
    codes |= (torch.randint(0, 2, codes.shape, generator=g) << 7).to(torch.uint8)
    rows = codes.numpy()
    if fmt == R.MX:
        rows[:, 512:528] = torch.randint(10, 247, (n, 16), generator=g).numpy()
        rows[:, 528:] = torch.randn(n, 64, generator=g).to(torch.bfloat16).view(torch.uint8).numpy().reshape(n, 128)
    return rows


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("lens,block", [([1], 64), ([0, 5, 0, 0, 17, 3], 4), ([130, 1, 64], 64), ([33] * 70, 7),
                                        ([3] * 1200, 1)])
@pytest.mark.parametrize("use_first", [False, True])
def test_gather_rows_bit_for_bit(use_first, lens, block, fmt):
    g = torch.Generator().manual_seed(len(lens) + fmt)
    first = [(5 * i) % 23 for i in range(len(lens))] if use_first else [0] * len(lens)
    pages = [-(-(n + f) // block) for n, f in zip(lens, first)]
    total = sum(pages) + 2
    raw = np.full((total * block, R.ROW_BYTES[fmt]), 0xFF, dtype=np.uint8)
    perm = torch.randperm(total, generator=g).tolist()
    table = np.full((len(lens), max(pages) + 1), -5, dtype=np.int32)
    want, at = [], 0
    for b, n in enumerate(lens):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
        rows = _good_rows(g, n, fmt)
        for i in range(n):
            k = first[b] + i
            raw[table[b, k // block] * block + k % block] = rows[i]
        want.append(rows)
    want = np.concatenate(want)
    n = want.shape[0]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    extra = 3
    wide = torch.full((n + extra, 584), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :576]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.mla_latent_cache_gather(_cache(raw, fmt, block), torch.from_numpy(table).cuda(), cu, n + extra, out=out,
                              first=torch.tensor(first, dtype=torch.int32, device="cuda") if use_first else None,
                              kv_scale=_kv_scale(fmt), status=status)
    got = out.cpu()
    assert int(status.item()) == 0
    assert (wide.cpu()[:, 576:] == 7.0).all() and (got[n:] == 7.0).all()  # rows behind the last sequence stay
    if fmt == R.E4M3:
        val = (R.LUT[want].astype(np.float32) * np.float32(SCALE)).astype(np.float32)
    else:
        val = R.values(want, fmt).astype(np.float32)
    assert np.array_equal(got[:n].contiguous().view(torch.int16).numpy().view(np.uint16), R.bf16_bits(val))


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_gather_leaves_out_what_does_not_exist(fmt):
    g = torch.Generator().manual_seed(1)
    block = 8
    raw = _good_rows(g, 4 * block, fmt)
    table = torch.tensor([[0, 99, 2], [-1, 1, 3]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 30, 50], dtype=torch.int32, device="cuda")  # sequence 0 is 6 rows longer than its table
    out = torch.full((60, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    L.mla_latent_cache_gather(_cache(raw, fmt, block), table, cu, 60, out=out, first=first, kv_scale=_kv_scale(fmt),
                              status=status)
    assert int(status.item()) == E.MLA_STATUS_SLOT_RANGE | E.MLA_STATUS_LEN_RANGE
    val = R.values(raw, fmt, SCALE)
    o = out.float().cpu().numpy()
    pages = {0: [0, None, 2], 1: [None, 1, 3]}
    for r in range(60):
        b = 0 if r < 30 else 1
        k = r if b == 0 else r - 30 + 4
        page = pages[b][k // block] if r < 50 and k < 24 else None
        if page is None:
            assert (o[r] == 3.0).all()
        else:
            assert np.allclose(o[r], val[page * block + k % block], rtol=2.0 ** -8, atol=1e-30)


# ---- attention -----------------------------------------------------------------------------

class _Case:
    """Sequences over a paged cache whose rows outside them are NaN."""

    def __init__(self, fmt, H, lens, prefixes=(), members=None, block=16, q8=False, seed=0, q_row=576, std=1.0,
                 pad_cols=2):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.H, self.lens, self.prefixes, self.block = fmt, H, list(lens), list(prefixes), block
        T = len(lens)
        self.members = members if members is not None else ([0, T] if prefixes else [0])
        pages = [-(-n // block) for n in self.prefixes + self.lens]
        total = sum(pages) + 2
        raw = np.full((total * block, R.ROW_BYTES[fmt]), 0xFF, dtype=np.uint8)
        perm = torch.randperm(total, generator=g).tolist()
        tables, self.keys, at = [], [], 0
        for n, m in zip(self.prefixes + self.lens, pages):
            pg = perm[at:at + m]
            at += m
            tables.append(pg)
            x = _bf(g, n, 576, std=std)
            kw = dict(kv_scale=SCALE) if fmt == R.E4M3 else {}
            rows = R.insert_rows(x[:, :512], x[:, 512:], fmt, **kw) if n else np.zeros((0, R.ROW_BYTES[fmt]), np.uint8)
            slot = np.array([pg[k // block] * block + k % block for k in range(n)], dtype=np.int64)
            raw[slot] = rows
            self.keys.append(R.values(rows, fmt, SCALE))
        self.cache = _cache(raw, fmt, block)

        def table(rows, cols):
            t = np.full((len(rows), cols), 2 ** 30, dtype=np.int32)  # entries behind the length are never followed
            for i, r in enumerate(rows):
                t[i, :len(r)] = r
            return torch.from_numpy(t).cuda()

        nP = len(self.prefixes)
        self.prefix_table = table(tables[:nP], max(map(len, tables[:nP])) + pad_cols) if nP else None
        self.prefix_lens = torch.tensor(self.prefixes, dtype=torch.int32, device="cuda") if nP else None
        self.offsets = torch.tensor(self.members, dtype=torch.int32, device="cuda") if nP else None
        self.table = table(tables[nP:], max(map(len, tables[nP:])) + pad_cols)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        q = _bf(g, T, H, q_row)[:, :, :576]
        self.q_scale = None
        if q8:
            raw_q = R.e4m3_bytes((q.float().numpy() / np.float32(SCALE)).astype(np.float64))
            self.q64 = R.LUT[raw_q] * float(np.float32(SCALE))
            buf = torch.zeros(T, H, q_row if q_row % 16 == 0 else 576, dtype=torch.uint8, device="cuda")
            buf[:, :, :576] = torch.from_numpy(raw_q).cuda()
            self.q, self.q_scale = buf[:, :, :576], torch.full((1,), SCALE, device="cuda")
        else:
            self.q64 = q.double().numpy()
            self.q = _move(q)
        self.sm_scale = 192 ** -0.5

    def keys_of(self, t):
        nP = len(self.prefixes)
        own = self.keys[nP + t]
        for g in range(nP):
            if self.members[g] <= t < self.members[g + 1]:
                return np.concatenate([self.keys[g], own])
        return own

    def call(self, **kw):
        return L.mla_prefix_decode_attention(
            self.q, self.cache, self.table, self.seq_lens, sm_scale=self.sm_scale, prefix_table=self.prefix_table,
            prefix_lens=self.prefix_lens, group_offsets=self.offsets, q_scale=self.q_scale,
            kv_scale=_kv_scale(self.fmt), **kw)

    def check(self, out, lse):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        f8 = self.fmt == R.E4M3 and self.q_scale is not None
        for t in range(len(self.lens)):
            o, s, tol, stol = R.attend(self.q64[t], self.keys_of(t), self.sm_scale, f8)
            bad = ~(np.abs(out[t] - o) <= tol)
            assert not bad.any(), (t, int(bad.sum()), np.abs(out[t] - o).max(), tol.max())
            if np.isinf(s).any():
                assert np.array_equal(lse[t], s), t
            else:
                assert (np.abs(lse[t] - s) <= stol).all(), (t, np.abs(lse[t] - s).max(), stol.max())


def _run(case, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cap = case.prefix_table.shape[1] * case.block if case.prefixes else 0
    need = E.mla_prefix_attend_workspace(len(case.lens), case.H, len(case.prefixes), cap)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN throughout
    out, lse = case.call(status=status, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    case.check(out, lse)
    return out, lse


KINDS = [(R.BF16, False), (R.BF16, True), (R.E4M3, False), (R.E4M3, True), (R.MX, False), (R.MX, True)]
KIND_IDS = [f"{NAMES[f]}-{'q8' if q else 'q16'}" for f, q in KINDS]


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("n", [1, 63, 64, 65, 128, 200, 1000])
def test_attend_one_token(n, fmt, q8):
    _run(_Case(fmt, 16, [n], q8=q8, seed=n))


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("H", [1, 3, 16, 63, 64, 65, 128, 130])
def test_attend_head_counts(H, fmt, q8):
    _run(_Case(fmt, H, [70, 5, 129], prefixes=[100], q8=q8, seed=H))


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
@pytest.mark.parametrize("block", [1, 2, 7, 16, 64, 100, 256])
def test_attend_block_sizes(block, fmt, q8):
    _run(_Case(fmt, 8, [70, 0, 300], prefixes=[130], block=block, q8=q8, seed=block))


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
def test_attend_prefix_for_many_tokens(fmt, q8):
    _run(_Case(fmt, 16, [(37 * i) % 90 for i in range(60)], prefixes=[700], q8=q8, seed=4))


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
def test_attend_groups(fmt, q8):
    """Several prefixes, an empty group, an empty prefix, tokens before the first group and behind the last."""
    _run(_Case(fmt, 5, [3, 0, 64, 10, 0, 1, 7, 0, 80, 2], prefixes=[65, 40, 0, 300], members=[1, 4, 4, 6, 9], q8=q8,
               seed=6))


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
def test_attend_rows_without_keys(fmt, q8):
    case = _Case(fmt, 16, [0, 0, 5, 0], q8=q8, seed=8)
    out, lse = _run(case)
    assert (out[[0, 1, 3]] == 0).all() and (lse[[0, 1, 3]] == float("-inf")).all()
    none = _Case(fmt, 16, [0, 0], prefixes=[0], q8=q8, seed=8)
    out, lse = _run(none)
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_attend_more_tokens_than_threads_and_empty_stretches():
    lens = [0] * 700
    for i in range(0, 700, 11):
        lens[i] = 1 + i % 130
    _run(_Case(R.E4M3, 4, lens, q8=True, seed=12))
    _run(_Case(R.BF16, 4, lens, prefixes=[90], members=[350, 600], seed=12))


def test_attend_long_context_over_all_ctas():
    _run(_Case(R.BF16, 16, [20000], block=64, seed=13))
    _run(_Case(R.MX, 2, [1, 9000], prefixes=[12345], block=64, seed=14))


def test_attend_strided_queries():
    _run(_Case(R.BF16, 16, [50, 60], prefixes=[64], q_row=640, seed=15))
    _run(_Case(R.E4M3, 16, [50, 60], prefixes=[64], q_row=640, q8=True, seed=15))


def test_attend_prefix_only():
    case = _Case(R.BF16, 16, [0] * 9, prefixes=[150], seed=16)
    case.table = case.seq_lens = None
    _run(case)


def test_attend_moving_maximum():
    """Scores that grow along the keys by far more than 2^8 a tile: the reference maximum moves again and again."""
    case = _Case(R.BF16, 16, [700, 64], prefixes=[500], seed=17, std=6.0)
    case.sm_scale = 1.0
    _run(case)


def test_attend_zero_scale_is_the_mean():
    case = _Case(R.BF16, 2, [100], seed=18)
    case.sm_scale = 0.0
    _run(case)


def test_attend_cuts_lengths_and_leaves_out_missing_pages():
    g = torch.Generator().manual_seed(2)
    block, fmt = 16, R.BF16
    rows = _good_rows(g, 8 * block, fmt)
    val = R.values(rows, fmt)
    cache = _cache(rows, fmt, block)
    q = _bf(g, 3, 16, 576)
    table = torch.tensor([[0, 1, 2], [3, 99, 4], [-7, 5, 6]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1000, 40, -3], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = L.mla_prefix_decode_attention(q.cuda(), cache, table, lens, sm_scale=0.07, status=status)
    assert int(status.item()) == E.MLA_STATUS_LEN_RANGE | E.MLA_STATUS_SLOT_RANGE
    keys = [val[:48], np.concatenate([val[48:64], val[64:72]]), val[:0]]
    for t in range(3):
        o, s, tol, stol = R.attend(q[t].double().numpy(), keys[t], 0.07)
        assert (np.abs(out[t].double().cpu().numpy() - o) <= tol).all()
        if t < 2:
            assert (np.abs(lse[t].double().cpu().numpy() - s) <= stol).all()
    # all of a sequence's pages missing: a row without keys
    lens = torch.tensor([16], dtype=torch.int32, device="cuda")
    out, lse = L.mla_prefix_decode_attention(q[:1].cuda(), cache, table[2:], lens, sm_scale=0.07)
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_attend_same_bits_every_time():
    case = _Case(R.MX, 16, [500, 20, 64, 3], prefixes=[900], seed=20)
    a = _run(case)
    for _ in range(3):
        b = _run(case)
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


# ---- together, as a decode step uses them -----------------------------------------------------

def _step(fmt, H, T, steps, prefix, block=16, norm=True):
    """Decode steps: a new row per token (insert), the epilogue's query rows, attention over prefix and own keys."""
    g = torch.Generator().manual_seed(31)
    scale = _kv_scale(fmt)
    per = -(-steps // block)
    n_blocks = -(-prefix // block) + T * per + 1
    raw = np.full((n_blocks * block, R.ROW_BYTES[fmt]), 0xFF, dtype=np.uint8)
    cache = _cache(raw, fmt, block)
    perm = torch.randperm(n_blocks, generator=g).to(torch.int32)
    n_pre = -(-prefix // block)
    ptab = perm[None, :n_pre].contiguous().cuda()
    btab = perm[n_pre:n_pre + T * per].view(T, per).contiguous().cuda()
    w = (1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16)
    tab = W.rope_table(prefix + steps)
    # the prompt, once
    kv, pe = _bf(g, prefix, 512), _bf(g, prefix, 64)
    pos = torch.arange(prefix, dtype=torch.int32)
    slots = (perm[pos.long() // block].long() * block + pos.long() % block)
    L.mla_latent_cache_insert(kv.cuda(), pe.cuda(), cache, slots.cuda(), norm_weight=w.cuda(), positions=pos.cuda(),
                              cos_sin=tab.cuda(), kv_scale=scale)
    # the prompt's rows read back are the rows attended to
    back = L.mla_latent_cache_gather(cache, ptab, torch.tensor([0, prefix], dtype=torch.int32, device="cuda"), prefix,
                                     kv_scale=scale)
    rows = R.insert_rows(kv, pe, fmt, norm_weight=w, positions=pos, cos_sin=tab, kv_scale=SCALE)
    pre = R.values(rows, fmt, SCALE)
    assert np.allclose(back.double().cpu().numpy(), pre, rtol=2.0 ** -8, atol=1e-30)
    own = [np.zeros((0, 576)) for _ in range(T)]
    for i in range(steps):
        ql, qp = _bf(g, T, H, 512), _bf(g, T, H, 64)
        kv, pe = _bf(g, T, 512), _bf(g, T, 64)
        pos = torch.full((T,), prefix + i, dtype=torch.int32)
        slots = btab[:, i // block].long() * block + i % block
        L.mla_latent_cache_insert(kv.cuda(), pe.cuda(), cache, slots, norm_weight=w.cuda(), positions=pos.cuda(),
                                  cos_sin=tab.cuda(), kv_scale=scale)
        # the query rows; every cache row is skipped (slot -1), it has been written above
        skip = torch.full((T,), -1, dtype=torch.int64, device="cuda")
        dummy = torch.empty((1, block, 576), dtype=torch.bfloat16, device="cuda")
        q = E.fused_mla_decode_q_concat_kv_cache_insert(
            ql.cuda(), qp.cuda(), kv.cuda(), pe.cuda(), dummy, skip, positions=pos.cuda(), cos_sin=tab.cuda())
        lens = torch.full((T,), i + 1, dtype=torch.int32, device="cuda")
        out, lse = L.mla_prefix_decode_attention(
            q, cache, btab, lens, prefix_table=ptab,
            prefix_lens=torch.tensor([prefix], dtype=torch.int32, device="cuda"), sm_scale=192 ** -0.5,
            kv_scale=scale, pdl=True)
        rows = R.insert_rows(kv, pe, fmt, norm_weight=w, positions=pos, cos_sin=tab, kv_scale=SCALE)
        new = R.values(rows, fmt, SCALE)
        q64 = q.double().cpu().numpy()
        for t in range(T):
            own[t] = np.concatenate([own[t], new[t:t + 1]])
            o, s, tol, stol = R.attend(q64[t], np.concatenate([pre, own[t]]), 192 ** -0.5)
            assert (np.abs(out[t].double().cpu().numpy() - o) <= tol).all()
            assert (np.abs(lse[t].double().cpu().numpy() - s) <= stol).all()


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_decode_steps_end_to_end(fmt):
    _step(fmt, H=16, T=5, steps=6, prefix=203, block=4)


def test_captured_step_replays_with_new_lengths():
    """A captured call reads lengths, tables and rows of its replay, and two graphs do not share a workspace."""
    case = _Case(R.BF16, 16, [100, 30], prefixes=[80], seed=40)
    other = _Case(R.E4M3, 16, [9, 333, 64], q8=True, seed=41)
    case.call(), other.call()
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1, l1 = case.call()
    with torch.cuda.graph(g2):
        o2, l2 = other.call()
    g1.replay(), g2.replay()
    torch.cuda.synchronize()
    case.check(o1, l1), other.check(o2, l2)
    case.seq_lens.copy_(torch.tensor([7, 0]))
    case.lens = [7, 0]
    case.keys[1], case.keys[2] = case.keys[1][:7], case.keys[2][:0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
    torch.cuda.synchronize()
    case.check(o1, l1), other.check(o2, l2)


def test_attend_negative_scale():
    case = _Case(R.BF16, 16, [130, 0, 70], prefixes=[100], seed=60)
    case.sm_scale = -0.05
    _run(case)
    case = _Case(R.E4M3, 16, [130, 0, 70], prefixes=[100], q8=True, seed=61)
    case.sm_scale = -0.05
    _run(case)


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
def test_attend_large_prefix_groups_of_many_rows(fmt, q8):
    """Groups large enough for decoded tiles (where rows are decoded), over pages that are and are not whole boxes."""
    lens = [(13 * i) % 50 for i in range(40)]
    for block in (64, 20):
        _run(_Case(fmt, 32, lens, prefixes=[300, 129], members=[0, 17, 40], block=block, q8=q8, seed=62 + block))


def test_attend_missing_page_in_a_large_prefix():
    for fmt, q8, block in ((R.MX, False, 64), (R.BF16, False, 64), (R.E4M3, True, 64), (R.BF16, False, 20)):
        case = _Case(fmt, 32, [3] * 20, prefixes=[6 * block], block=block, q8=q8, seed=70)
        case.prefix_table[0, 2] = -1
        case.keys[0] = np.delete(case.keys[0], np.s_[2 * block:3 * block], axis=0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = case.call(status=status)
        case.check(out, lse)
        assert int(status.item()) == E.MLA_STATUS_SLOT_RANGE


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
def test_attend_values_at_the_ends_of_the_types(fmt, q8):
    """NaN and infinite latents reach exactly the tokens that attend to them."""
    case = _Case(fmt, 16, [70, 65, 5], q8=q8, seed=80)
    raw = case.cache.view(torch.uint8).view(-1, R.ROW_BYTES[fmt])
    page = int(case.table[1, 0])
    slot = page * case.block + 3  # token 1, key 3: value 7 becomes NaN
    if fmt == R.BF16:
        raw[slot].view(torch.bfloat16)[7] = float("nan")
    else:
        raw[slot, 7] = 0x7F
    out, lse = case.call()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    case.lens, out, lse = [70, 0, 5], out.clone(), lse.clone()
    out[1], lse[1] = 0, float("-inf")
    case.keys[1] = case.keys[1][:0]
    case.check(out, lse)


def test_attend_codes_of_every_value():
    """All finite e4m3 codes and a wide range of scale exponents through the decoding."""
    g = torch.Generator().manual_seed(90)
    for fmt, q8 in ((R.E4M3, True), (R.E4M3, False), (R.MX, False)):
        n, block = 256, 64
        raw = _good_rows(g, n, fmt)
        if fmt == R.MX:
            raw[:, 512:528] = torch.randint(100, 140, (n, 16), generator=g).numpy()
            raw[:, 512:514] = torch.randint(134, 136, (n, 2), generator=g).numpy()
        val = R.values(raw, fmt, 1.0)
        q = _bf(g, 1, 16, 576, std=0.01)
        if q8:
            qr = R.e4m3_bytes((q.float().numpy() / np.float32(SCALE)).astype(np.float64))
            qd, qs, q64 = torch.from_numpy(qr).cuda(), torch.full((1,), SCALE, device="cuda"), R.LUT[qr] * float(np.float32(SCALE))
        else:
            qd, qs, q64 = q.cuda(), None, q.double().numpy()
        scale = 2.0 ** -10
        out, lse = L.mla_prefix_decode_attention(
            qd, _cache(raw, fmt, block), torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.tensor([n], dtype=torch.int32, device="cuda"),
            sm_scale=scale, q_scale=qs, kv_scale=torch.ones(1, device="cuda") if fmt == R.E4M3 else None)
        o, s, tol, stol = R.attend(q64[0], val, scale, q8)
        assert (np.abs(out[0].double().cpu().numpy() - o) <= tol).all()
        assert (np.abs(lse[0].double().cpu().numpy() - s) <= stol).all()


def test_torch_forms_reject_wrong_tensors():
    case = _Case(R.BF16, 4, [5, 6], prefixes=[20], seed=95)
    good = dict(sm_scale=1.0, prefix_table=case.prefix_table, prefix_lens=case.prefix_lens)
    call = L.mla_prefix_decode_attention
    q, c, t, n = case.q, case.cache, case.table, case.seq_lens
    for args, kw in (((q.float(), c, t, n), {}), ((q[..., :575], c, t, n), {}), ((q, c[..., :575], t, n), {}),
                     ((q, c, t.long(), n), {}), ((q, c, t[:1], n), {}), ((q, c, t, n.long()), {}), ((q, c, t, None), {}),
                     ((q, c, t.cpu(), n), {}), ((q, c, t, n), dict(kv_scale=torch.ones(1, device="cuda"))),
                     ((q, c, t, n), dict(q_scale=torch.ones(1, device="cuda"))),
                     ((q, c, t, n), dict(prefix_lens=None)), ((q, c, t, n), dict(prefix_table=None)),
                     ((q, c, t, n), dict(group_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))),
                     ((q, c, t, n), dict(out=torch.empty((2, 4, 512), device="cuda"))),
                     ((q, c, t, n), dict(lse=torch.empty((2, 5), device="cuda"))),
                     ((q, c, t, n), dict(status=torch.zeros(2, dtype=torch.int32, device="cuda")))):
        with pytest.raises(ValueError):
            call(*args, **{**good, **kw})
    with pytest.raises(E.MlaError):  # too small a workspace
        call(q, c, t, n, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), **good)
    x, pe = torch.zeros((3, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    for args, kw in (((x.float(), pe, c, slots), {}), ((x, pe[:2], c, slots), {}), ((x, pe, c, slots.int()), {}),
                     ((x, pe, c, slots), dict(norm_weight=torch.ones(512, device="cuda"))),
                     ((x, pe, c, slots), dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda"))),
                     ((x.t().contiguous().t(), pe, c, slots), {})):
        with pytest.raises(ValueError):
            L.mla_latent_cache_insert(*args, **kw)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    for args, kw in (((c, t, cu[:2], 4), {}), ((c, t, cu.long(), 4), {}), ((c, t, cu, 4), dict(first=cu)),
                     ((c, t, cu, 4), dict(out=torch.empty((5, 576), dtype=torch.bfloat16, device="cuda")))):
        with pytest.raises(ValueError):
            L.mla_latent_cache_gather(*args, **kw)


def test_calls_on_two_streams_at_once():
    a = _Case(R.BF16, 16, [600, 64, 3], prefixes=[500], seed=50)
    b = _Case(R.MX, 16, [64, 800], seed=51)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        got.append((a, a.call(stream=s1)))
        got.append((b, b.call(stream=s2)))
    torch.cuda.synchronize()
    for c, (o, l) in got:
        c.check(o, l)


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
def test_attend_many_short_sequences(fmt, q8):
    """A dozen or more pieces of work for every SM, of none to four tiles each, some behind a prefix."""
    lens = [(53 * i) % 211 if i % 5 else 0 for i in range(1800)]
    _run(_Case(fmt, 4, lens, prefixes=[70, 130], members=[0, 31, 900], block=32, q8=q8, seed=40))


def test_attend_one_query_for_all_heads():
    """Queries broadcast over the heads (stride 0)."""
    case = _Case(R.BF16, 20, [70, 130], prefixes=[64], seed=41)
    case.q = case.q[:, :1].expand(-1, 20, -1)
    case.q64 = np.repeat(case.q64[:, :1], 20, axis=1)
    out, _ = _run(case)
    assert (out == out[:, :1]).all()


@pytest.mark.parametrize("fmt,q8", KINDS, ids=KIND_IDS)
def test_attend_the_same_pages_twice(fmt, q8):
    """A sequence whose table names a page several times, and sequences that share their pages."""
    for block in (16, 64):
        case = _Case(fmt, 16, [2 * block, 4 * block + 5], block=block, q8=q8, seed=42)
        pages, keys = case.table[0, :2].tolist(), case.keys[0]
        order = [0, 0, 1, 0, 0]
        case.table[1, :5] = torch.tensor([pages[i] for i in order], dtype=torch.int32)
        case.keys[1] = np.concatenate([keys[i * block:(i + 1) * block] for i in order])[:4 * block + 5]
        _run(case)


def test_attend_long_stretches_of_tokens_without_keys():
    """Half a million tokens, a few of which have keys."""
    g = torch.Generator().manual_seed(43)
    T, block = 500_000, 16
    rows = _good_rows(g, 8 * block, R.BF16)
    val = R.values(rows, R.BF16)
    q = torch.zeros((T, 1, 576), dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(T, dtype=torch.int32, device="cuda")
    picked = [0, 1, 31, 70_000, 70_001, 400_032, T - 1]
    some = _bf(g, len(picked), 1, 576)
    for i, t in enumerate(picked):
        lens[t], q[t] = 3 + 17 * i, some[i].cuda()
    lens[5] = -4
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None].expand(T, 8)
    out, lse = L.mla_prefix_decode_attention(q, _cache(rows, R.BF16, block), table, lens, sm_scale=0.07)
    for i, t in enumerate(picked):
        o, s, tol, stol = R.attend(some[i].double().numpy(), val[:3 + 17 * i], 0.07)
        assert (np.abs(out[t].double().cpu().numpy() - o) <= tol).all(), t
        assert (np.abs(lse[t].double().cpu().numpy() - s) <= stol).all(), t
    lse[picked], out[picked] = float("-inf"), 0
    assert (lse == float("-inf")).all() and (out == 0).all()


@pytest.mark.parametrize("fmt,q8", [(R.BF16, False), (R.E4M3, True), (R.MX, False)], ids=["bf16", "e4m3", "mx"])
def test_cache_of_more_than_32_bits(fmt, q8):
    """Rows beyond byte 2^32 of the cache: written, read back and attended to."""
    block, n = 64, 200
    blocks = 2 ** 32 // (block * R.ROW_BYTES[fmt]) + 8
    case = _Case(fmt, 16, [n], block=block, q8=q8, seed=44)
    small = case.cache.view(torch.uint8).view(-1, block, R.ROW_BYTES[fmt])
    big = torch.full((blocks, block, R.ROW_BYTES[fmt]), 0xFF, dtype=torch.uint8, device="cuda")
    big[-small.shape[0]:] = small
    assert (blocks - small.shape[0]) * block * R.ROW_BYTES[fmt] > 2 ** 32 - 2 ** 20
    want = case.call()
    near = L.mla_latent_cache_gather(case.cache, case.table[:, :4], torch.tensor([0, n], dtype=torch.int32, device="cuda"), n,
                                     kv_scale=_kv_scale(fmt))
    case.cache = big.view(torch.bfloat16) if fmt == R.BF16 else big
    case.table[:, :4] += blocks - small.shape[0]
    got = _run(case)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    far = L.mla_latent_cache_gather(case.cache, case.table[:, :4], torch.tensor([0, n], dtype=torch.int32, device="cuda"), n,
                                    kv_scale=_kv_scale(fmt))
    assert torch.equal(far.view(torch.int16), near.view(torch.int16))
    x = _bf(torch.Generator().manual_seed(45), 3, 576).cuda()
    slots = torch.arange(blocks * block - 3, blocks * block, device="cuda")
    tiny = torch.zeros((1, block, R.ROW_BYTES[fmt]), dtype=torch.uint8, device="cuda")
    tiny = tiny.view(torch.bfloat16) if fmt == R.BF16 else tiny
    for cache, at in ((case.cache, slots), (tiny, torch.arange(3, device="cuda"))):
        L.mla_latent_cache_insert(x[:, :512], x[:, 512:], cache, at, kv_scale=_kv_scale(fmt))
    assert torch.equal(case.cache.view(torch.uint8)[-1, -3:], tiny.view(torch.uint8)[0, :3])
