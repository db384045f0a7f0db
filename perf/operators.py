"""The latent-cache operators, their plain forms and the cases they are measured at.

Three operators around the paged latent KV cache of MLA decode (a row holds
512 latent values and 64 rotary values):

insert  one latent row per token into the cache, in one pass: optional RMS norm
        of the 512 latents, optional rotation of the 64 rotary values, then a
        bf16 row, e4m3 bytes of x / scale, or a microscaled row (e4m3 codes
        with one power-of-two scale for each 32 latents, rotary part in bf16);
gather  rows of paged sequences read back as contiguous bf16 rows;
attend  decode attention of T query tokens with H heads over the paged cache;
        the tokens share one long prefix, whose keys come once for all, and
        each has keys of its own behind it.

Cache rows by format: "bf16" 576 values, "e4m3" 576 bytes with one scale for
the whole cache, "mx" 656 bytes: 512 codes, 16 scale exponents (2^(byte - 127)),
64 bf16 rotary values.
"""

import math
import random

import torch

own = False

PE = 64
NOPE = 512
ROW = NOPE + PE
GROUP = 32                      # latents that share one scale of an "mx" row
MX_ROW = NOPE + NOPE // GROUP + 2 * PE
MX_EXP = (-117, 119)            # exponents a scale may take
E4M3_MAX = 448.0
SM_SCALE = 1.0 / math.sqrt(192.0)  # 128 nope + 64 rotary dims of a head before absorption
EPS = 1e-6
DEV = "cuda"

_ROW_BYTES = {"bf16": 2 * ROW, "e4m3": ROW, "mx": MX_ROW}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def _insert(name, T, fmt, norm=True, rope=True, row=NOPE, rope_rows=32768, block=64):
    return {"name": name, "op": "insert", "T": T, "fmt": fmt, "norm": norm, "rope": rope, "row": row,
            "rope_rows": rope_rows, "block": block}


def _gather(name, seqs, lo, hi, fmt, lens=0, block=64, first=False):
    return {"name": name, "op": "gather", "seqs": seqs, "lo": lo, "hi": hi, "fmt": fmt, "lens": lens, "block": block,
            "first": first}


def _attend(name, T, H, prefix, lo, hi, fmt, q8=False, lens=0, block=64):
    return {"name": name, "op": "attend", "T": T, "H": H, "prefix": prefix, "lo": lo, "hi": hi, "fmt": fmt, "q8": q8,
            "lens": lens, "block": block}


def listed():
    return [
        # one decode step of a single sequence: the new token's row
        _insert("insert_t1_mx", 1, "mx"),
        # one decode step of an odd-sized batch into a per-tensor e4m3 cache
        _insert("insert_t65_e4m3", 65, "e4m3"),
        # the latents as a column slice of a wider projection output, already normalised by the model
        _insert("insert_t1024_mx_strided", 1024, "mx", norm=False, row=1536),
        # the prompt tokens of a large batch, long-context rotary table
        _insert("insert_t8192_mx", 8192, "mx", rope_rows=131072),
        # the cached context of a few short requests
        _gather("gather_5_short_mx", 5, 1, 300, "mx", lens=1, block=16),
        # chunks of long contexts, from a position inside each sequence on
        _gather("gather_16_long_mx", 16, 2048, 8192, "mx", lens=2, first=True),
        _gather("gather_32_long_e4m3", 32, 1024, 8192, "e4m3", lens=3),
        # a single sequence's decode step, the latency case
        _attend("attend_t1_h16_bf16", 1, 16, 0, 1000, 1000, "bf16"),
        # a decode batch behind a common system prompt, 16 heads (one of 8 tensor-parallel ranks)
        _attend("attend_t64_h16_prefix_e4m3", 64, 16, 8192, 0, 512, "e4m3", q8=True, lens=4),
        # all 128 heads on one card, odd prefix
        _attend("attend_t16_h128_prefix_bf16", 16, 128, 16001, 1, 2048, "bf16", lens=5),
        # long ragged contexts without a prefix: bound by reading the cache
        _attend("attend_t32_h16_long_e4m3", 32, 16, 0, 4096, 32768, "e4m3", q8=True, lens=6),
        # many requests over one long document
        _attend("attend_t256_h16_document_mx", 256, 16, 32768, 1, 256, "mx", lens=7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    fmt = rng.choice(["bf16", "e4m3", "mx", "mx"])
    block = rng.choice([16, 32, 64, 64, 128, 20])
    op = rng.choice(["insert", "gather", "attend", "attend"])
    if op == "insert":
        return {k: v for k, v in _insert("", _log(rng, 1, 8192), fmt, norm=rng.random() < 0.7, rope=rng.random() < 0.8,
                                         row=rng.choice([NOPE, ROW, 1536]),
                                         rope_rows=rng.choice([32768, 131072]), block=block).items() if k != "name"}
    if op == "gather":
        hi = _log(rng, 1, 6000)
        return {k: v for k, v in _gather("", _log(rng, 1, 24), _log(rng, 1, hi), hi, fmt, lens=rng.randrange(1 << 20),
                                         block=block, first=rng.random() < 0.5).items() if k != "name"}
    H = rng.choice([1, 8, 16, 16, 32, 128])
    T = _log(rng, 1, max(1, 4096 // max(H, 16)))
    prefix = 0 if rng.random() < 0.25 else _log(rng, 64, 32000)
    hi = _log(rng, 1, max(2, min(16384, 400000 // T)))
    return {k: v for k, v in _attend("", T, H, prefix, rng.choice([0, 1, max(1, hi // 2)]), hi, fmt,
                                     q8=fmt == "e4m3" and rng.random() < 0.7, lens=rng.randrange(1 << 20),
                                     block=block).items() if k != "name"}


def _lens(case):
    """The sequence lengths of a gather or attend case."""
    r = random.Random("lens %d" % case["lens"])
    n = case["seqs"] if case["op"] == "gather" else case["T"]
    return [r.randint(case["lo"], case["hi"]) for _ in range(n)]


def _firsts(case):
    """The position each sequence of a gather case is read from."""
    r = random.Random("first %d" % case["lens"])
    return [r.randint(0, 500) if case["first"] else 0 for _ in range(case["seqs"])]


def work(case):
    row = _ROW_BYTES[case["fmt"]]
    if case["op"] == "insert":
        T = case["T"]
        per = 2 * ROW + 8 + row + (4 + 4 * PE if case["rope"] else 0)
        return {"bytes": T * per + (2 * NOPE if case["norm"] else 0), "flops": T * NOPE * (7 if case["norm"] else 3)}
    if case["op"] == "gather":
        n = sum(_lens(case))
        return {"bytes": n * (row + 2 * ROW), "flops": n * ROW}
    T, H, lens = case["T"], case["H"], _lens(case)
    keys = case["prefix"] + sum(lens)
    bytes_ = T * H * (ROW * (1 if case["q8"] else 2) + 2 * NOPE + 4) + keys * row
    return {"bytes": bytes_, "flops": 2 * (ROW + NOPE) * H * (T * case["prefix"] + sum(lens))}


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------

def _group_exponents(y):
    """The scale exponent of each group of 32 of y [n, 512]: the least e with max |y| <= 448 * 2^e, over the finite
    values."""
    a = y.abs().reshape(y.shape[0], -1, GROUP)
    a = torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax(-1)
    m, e = torch.frexp(a)  # a = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = e.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)
    return torch.where(a > 0, e, torch.full_like(e, MX_EXP[0])).clamp(*MX_EXP)


def _pow2(e, dtype):
    """2^e for integers e, in two factors so that neither leaves the type's range."""
    h = torch.div(e, 2, rounding_mode="floor")
    one = torch.ones((), dtype=dtype, device=e.device)
    return torch.ldexp(one, h) * torch.ldexp(one, e - h)


def _e4m3(x):
    """e4m3 bytes of x, ties to even, beyond 448 to +-448."""
    return x.float().clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _rotate(pe, positions, table):
    c = table[positions.long()]
    cos, sin = c[:, :PE // 2], c[:, PE // 2:]
    a, b = pe[:, :PE // 2], pe[:, PE // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], 1)


def _encode(y, pe, fmt, scale):
    """Cache rows, as bytes [n, row bytes], of the latents y and the rotary values pe."""
    if fmt == "bf16":
        return torch.cat([y, pe], 1).to(torch.bfloat16).view(torch.uint8)
    if fmt == "e4m3":
        return _e4m3(torch.cat([y, pe], 1).float() / scale)
    e = _group_exponents(y)
    codes = _e4m3((y.reshape(y.shape[0], -1, GROUP) * _pow2(-e, y.dtype)[..., None]).reshape(y.shape[0], NOPE))
    return torch.cat([codes, (e + 127).to(torch.uint8), pe.to(torch.bfloat16).contiguous().view(torch.uint8)], 1)


def _decode(rows, fmt, scale):
    """fp32 values [n, 576] of cache rows given as bytes [..., row bytes]."""
    if fmt == "bf16":
        return rows.view(torch.bfloat16).float()
    if fmt == "e4m3":
        return rows.view(torch.float8_e4m3fn).float() * scale
    codes = rows[..., :NOPE].view(torch.float8_e4m3fn).float()
    e = rows[..., NOPE:NOPE + NOPE // GROUP].to(torch.int32) - 127
    pe = rows[..., NOPE + NOPE // GROUP:].contiguous().view(torch.bfloat16).float()
    return torch.cat([codes * _pow2(e, torch.float32).repeat_interleave(GROUP, -1), pe], -1)


def _as_bytes(cache):
    return cache.view(torch.uint8).view(-1, cache.shape[-1] * cache.element_size())


def _plain_insert(s):
    x = s["kv_c"].double() if s["norm"] is not None else s["kv_c"].float()
    if s["norm"] is not None:  # 64 bits: a value next to a border of its code must fall on the right side
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["norm"].double()
    pe = s["k_pe"].float()
    if s["cos_sin"] is not None:
        pe = _rotate(pe, s["positions"], s["cos_sin"])
    if s["fmt"] != "mx":
        x = x.float()
    _as_bytes(s["cache"])[s["slots"]] = _encode(x, pe, s["fmt"], s["kv_scale"])


def _plain_gather(s):
    n = s["rows"]
    r = torch.arange(n, device=DEV)
    b = torch.searchsorted(s["cu"].long(), r, right=True) - 1
    k = r - s["cu"].long()[b] + (s["first"].long()[b] if s["first"] is not None else 0)
    bs = s["cache"].shape[1]
    slot = s["table"].long()[b, k // bs] * bs + k % bs
    return _decode(_as_bytes(s["cache"])[slot], s["fmt"], s["kv_scale"]).to(torch.bfloat16)


def _plain_attend(s):
    q = s["q"].view(torch.float8_e4m3fn).float() * s["q_scale"] if s["q_scale"] is not None else s["q"].float()
    T, H, bs, rows = q.shape[0], q.shape[1], s["cache"].shape[1], _as_bytes(s["cache"])
    scores, values = [], []
    if s["prefix_lens"] is not None:
        k = torch.arange(s["prefix"], device=DEV)
        kv = _decode(rows[s["prefix_table"].long()[0, k // bs] * bs + k % bs], s["fmt"], s["kv_scale"])
        scores.append((q.reshape(T * H, ROW) @ kv.t()).view(T, H, -1) * SM_SCALE)
        values.append(kv[:, :NOPE])
    k = torch.arange(s["longest"], device=DEV)
    kv = _decode(rows[s["table"].long()[:, k // bs] * bs + k % bs], s["fmt"], s["kv_scale"])
    live = k < s["lens"][:, None]
    own_scores = torch.einsum("thd,tkd->thk", q, kv) * SM_SCALE
    scores.append(own_scores.masked_fill(~live[:, None, :], float("-inf")))
    values.append(torch.where(live[..., None], kv[..., :NOPE], torch.zeros_like(kv[..., :NOPE])))
    x = torch.cat(scores, -1)
    top = x.amax(-1, keepdim=True) if x.shape[-1] else x.new_full((T, H, 1), float("-inf"))
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("thk,tkd->thd", p[..., x.shape[-1] - s["longest"]:], values[-1])
    if s["prefix_lens"] is not None:
        out = out + (p[..., :s["prefix"]].reshape(T * H, -1) @ values[0]).view(T, H, NOPE)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out.to(torch.bfloat16), (torch.log(total) + top).squeeze(-1)


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

def _table(rows):
    p = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None]
    w = 10000.0 ** (-torch.arange(PE // 2, dtype=torch.float64, device=DEV) / (PE // 2))
    return torch.cat([torch.cos(p * w), torch.sin(p * w)], 1).float()


def _cache_of(g, n_blocks, block, fmt, scale):
    """A cache whose rows hold N(0, 1) latents and rotary values."""
    n = n_blocks * block
    out = torch.empty((n, _ROW_BYTES[fmt]), dtype=torch.uint8, device=DEV)
    for i in range(0, n, 1 << 17):
        m = min(1 << 17, n - i)
        x = torch.randn((m, ROW), generator=g, device=DEV).to(torch.bfloat16).float()
        out[i:i + m] = _encode(x[:, :NOPE], x[:, NOPE:], fmt, scale)
    out = out.view(n_blocks, block, -1)
    return out.view(torch.bfloat16) if fmt == "bf16" else out


def _pages(g, lens, block, perm, at):
    """Page numbers [len(lens), most pages] of sequences of these lengths, taken from `perm` from `at` on."""
    need = torch.tensor([-(-n // block) for n in lens])
    cols = max(1, int(need.max()) if len(lens) else 1)
    start = torch.cumsum(need, 0) - need + at
    j = torch.arange(cols)
    idx = torch.where(j < need[:, None], start[:, None] + j, torch.zeros((), dtype=torch.long))
    return perm[idx.to(DEV)].to(torch.int32), at + int(need.sum())


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    fmt, block = case["fmt"], case["block"]
    scale = torch.full((1,), 0.05, device=DEV) if fmt == "e4m3" else None
    s = {"op": case["op"], "fmt": fmt, "kv_scale": scale}

    def bf(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    if case["op"] == "insert":
        T = case["T"]
        n_blocks = -(-5 * T // (4 * block)) + 1
        off = 512 if case["row"] >= 2 * NOPE else 0
        s["kv_c"] = (bf(T, case["row"]) * (2.0 if case["norm"] else 1.0))[:, off:off + NOPE]
        s["k_pe"] = bf(T, PE)
        s["norm"] = (1.0 + 0.1 * bf(NOPE)).to(torch.bfloat16) if case["norm"] else None
        s["slots"] = torch.randperm(n_blocks * block, generator=g, device=DEV)[:T]
        s["cos_sin"] = _table(case["rope_rows"]) if case["rope"] else None
        s["positions"] = torch.randint(0, case["rope_rows"], (T,), generator=g, device=DEV, dtype=torch.int32)
        s["cache"] = torch.zeros((n_blocks, block, _ROW_BYTES[fmt]), dtype=torch.uint8, device=DEV)
        if fmt == "bf16":
            s["cache"] = s["cache"].view(torch.bfloat16)
        return s

    lens = _lens(case)
    if case["op"] == "gather":
        first = _firsts(case)
        ends = [n + f for n, f in zip(lens, first)]
        n_blocks = sum(-(-n // block) for n in ends) + 1
        perm = torch.randperm(n_blocks, generator=g, device=DEV)
        s["table"], _ = _pages(g, ends, block, perm, 0)
        s["first"] = torch.tensor(first, dtype=torch.int32, device=DEV) if case["first"] else None
        s["cu"] = torch.cumsum(torch.tensor([0] + lens), 0).to(torch.int32).to(DEV)
        s["rows"] = sum(lens)
    else:
        T, H = case["T"], case["H"]
        n_blocks = -(-case["prefix"] // block) + sum(-(-n // block) for n in lens) + 1
        perm = torch.randperm(n_blocks, generator=g, device=DEV)
        s["prefix"], s["prefix_table"], s["prefix_lens"], at = case["prefix"], None, None, 0
        if case["prefix"]:
            s["prefix_table"], at = _pages(g, [case["prefix"]], block, perm, 0)
            s["prefix_lens"] = torch.tensor([case["prefix"]], dtype=torch.int32, device=DEV)
        s["table"], _ = _pages(g, lens, block, perm, at)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["longest"] = max(lens)
        q = bf(T, H, ROW)
        s["q_scale"] = torch.full((1,), 0.05, device=DEV) if case["q8"] else None
        s["q"] = _e4m3(q.float() / s["q_scale"]) if case["q8"] else q
    s["cache"] = _cache_of(g, n_blocks, block, fmt, scale)
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def _cache_out(cache, fmt):
    """The cache as the numbers it holds, without a copy."""
    if fmt == "bf16":
        return {"rows": cache}
    if fmt == "e4m3":
        return {"codes": cache.view(torch.float8_e4m3fn)}
    return {"codes": cache[..., :NOPE].view(torch.float8_e4m3fn),
            "scales": cache[..., NOPE:NOPE + NOPE // GROUP].view(torch.float8_e8m0fnu),
            "pe": cache[..., NOPE + NOPE // GROUP:].view(torch.bfloat16)}


def run(state):
    s = state
    if s["op"] == "insert":
        if own:
            from mla_decode_attention_10_b200 import latent
            latent.mla_latent_cache_insert(
                s["kv_c"], s["k_pe"], s["cache"], s["slots"], norm_weight=s["norm"], eps=EPS,
                positions=s["positions"] if s["cos_sin"] is not None else None, cos_sin=s["cos_sin"],
                kv_scale=s["kv_scale"])
        else:
            _plain_insert(s)
        return _cache_out(s["cache"], s["fmt"])
    if s["op"] == "gather":
        if own:
            from mla_decode_attention_10_b200 import latent
            return latent.mla_latent_cache_gather(s["cache"], s["table"], s["cu"], s["rows"], first=s["first"],
                                                  kv_scale=s["kv_scale"])
        return _plain_gather(s)
    if own:
        from mla_decode_attention_10_b200 import latent
        out, lse = latent.mla_prefix_decode_attention(
            s["q"], s["cache"], s["table"], s["lens"], prefix_table=s["prefix_table"], prefix_lens=s["prefix_lens"],
            sm_scale=SM_SCALE, q_scale=s["q_scale"], kv_scale=s["kv_scale"])
    else:
        out, lse = _plain_attend(s)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------

def _e4m3_values():
    """The 256 values of e4m3 bytes: sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinity."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.nan if b & 0x7F == 0x7F else math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        v.append(-x if b & 0x80 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _nearest_e4m3(x):
    """x (64 bits) rounded to the nearest e4m3 value, ties to even, at most 448 in magnitude."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    e = e - (torch.exp2(e) > a.clamp(min=2.0 ** -6)).double() + (torch.exp2(e + 1) <= a).double()
    step = torch.exp2(e - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)  # torch.round: ties to even


def _values64(cache, fmt, scale, idx):
    raw = cache.view(torch.uint8).reshape(-1, _ROW_BYTES[fmt])[idx]
    if fmt == "bf16":
        return raw.view(torch.bfloat16).double()
    lut = _e4m3_values()
    if fmt == "e4m3":
        return lut[raw.long()] * scale.double()
    x = lut[raw[:, :NOPE].long()].view(-1, NOPE // GROUP, GROUP)
    x = x * torch.exp2(raw[:, NOPE:NOPE + NOPE // GROUP].double() - 127.0)[:, :, None]
    pe = raw[:, NOPE + NOPE // GROUP:].contiguous().view(torch.bfloat16).double()
    return torch.cat([x.reshape(-1, NOPE), pe], 1)


def _exact_insert(s):
    fmt, n = s["fmt"], s["cache"].shape[0] * s["cache"].shape[1]
    shape = s["cache"].shape[:2]
    x = s["kv_c"].double()
    if s["norm"] is not None:
        x = x / torch.sqrt((x * x).sum(1, keepdim=True) / NOPE + EPS) * s["norm"].double()
    pe = s["k_pe"].double()
    if s["cos_sin"] is not None:
        t = s["cos_sin"].double()[s["positions"].long()]
        pe = torch.stack([pe[:, j] * t[:, j] - pe[:, j + 32] * t[:, j + 32] if j < 32
                          else pe[:, j] * t[:, j - 32] + pe[:, j - 32] * t[:, j] for j in range(PE)], 1)

    def placed(rows):
        full = torch.zeros((n, rows.shape[1]), dtype=torch.float64, device=DEV)
        full[s["slots"]] = rows
        return full.view(*shape, -1)

    if fmt == "bf16":
        return {"rows": placed(torch.cat([x, pe], 1))}
    if fmt == "e4m3":
        return {"codes": placed(_nearest_e4m3(torch.cat([x, pe], 1) / s["kv_scale"].double()))}
    big = x.abs().view(-1, NOPE // GROUP, GROUP).amax(-1)
    e = torch.ceil(torch.log2((big / E4M3_MAX).clamp(min=2.0 ** MX_EXP[0])))
    e = e + (torch.exp2(e) * E4M3_MAX < big).double() - (torch.exp2(e - 1) * E4M3_MAX >= big).double()
    e = e.clamp(*MX_EXP)
    codes = _nearest_e4m3((x.view(-1, NOPE // GROUP, GROUP) / torch.exp2(e)[..., None]).reshape(-1, NOPE))
    scales = placed(torch.exp2(e))
    scales[(torch.ones(n, device=DEV).index_fill(0, s["slots"], 0.0) > 0).view(*shape)] = 2.0 ** -127  # byte 0
    return {"codes": placed(codes), "scales": scales, "pe": placed(pe)}


def _slots_of(table_row, first, n, block):
    k = torch.arange(first, first + n, device=DEV)
    return table_row.long()[k // block] * block + k % block


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "insert":
        return _exact_insert(s)
    lens, block = _lens(case), case["block"]
    if case["op"] == "gather":
        first = _firsts(case)
        idx = torch.cat([_slots_of(s["table"][i], first[i], n, block) for i, n in enumerate(lens)])
        return _values64(s["cache"], s["fmt"], s["kv_scale"], idx)
    T, H = case["T"], case["H"]
    q = s["q"].double() if s["q_scale"] is None else _e4m3_values()[s["q"].long()] * s["q_scale"].double()
    pre = None
    if case["prefix"]:
        pre = _values64(s["cache"], s["fmt"], s["kv_scale"], _slots_of(s["prefix_table"][0], 0, case["prefix"], block))
    out, lse = [], []
    for t in range(T):
        kv = _values64(s["cache"], s["fmt"], s["kv_scale"], _slots_of(s["table"][t], 0, lens[t], block))
        if pre is not None:
            kv = torch.cat([pre, kv])
        if kv.shape[0] == 0:
            out.append(torch.zeros((H, NOPE), dtype=torch.float64, device=DEV))
            lse.append(torch.full((H,), -math.inf, dtype=torch.float64, device=DEV))
            continue
        x = (q[t] @ kv.t()) * SM_SCALE
        lse.append(torch.logsumexp(x, 1))
        out.append(torch.exp(x - lse[-1][:, None]) @ kv[:, :NOPE])
    return {"out": torch.stack(out), "lse": torch.stack(lse)}
