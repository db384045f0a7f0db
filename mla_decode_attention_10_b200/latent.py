"""Torch-tensor form of the latent-cache operators of ``include/mla_epilogue.h``.

* ``mla_latent_cache_insert``: latent rows into the paged cache, with the norm,
  the rotation and the quantisation in the same pass;
* ``mla_latent_cache_gather``: rows of paged sequences read back as bf16;
* ``mla_prefix_decode_attention``: decode attention over the cache for a batch
  whose tokens share long prefixes.

The row format follows from the cache tensor: bf16 ``[num_blocks, block_size,
576]``; uint8 ``[..., 576]`` for e4m3 bytes with one ``kv_scale``; uint8
``[..., 656]`` for microscaled rows (512 e4m3 codes, 16 scale exponents, 64
bf16 rotary values).

Work is enqueued on ``stream``, or on the current stream of the tensors'
device.  Outputs and workspaces that are not given come from torch's
allocator on that stream.  Wrong arguments raise ``ValueError`` here or
``MlaError`` in the library; there is no fallback path.
"""

from __future__ import annotations

import functools
from typing import Optional, Tuple

import torch

from . import epilogue as E

# A decode step makes these calls once a layer, so the host side of a call
# counts: the checks compare integers and interned objects, and a device or
# stream is only entered when it is not the current one.

_BF16, _U8, _I32, _I64, _F32 = torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float32


def _fail(name: str, t: torch.Tensor, index: int, dtype: torch.dtype, shape: tuple) -> None:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.get_device() != index or t.dtype != dtype:
        raise ValueError(f"{name}: a {dtype} tensor on cuda:{index} is required, got {t.dtype} on {t.device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {list(shape)} is required, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _flat(name: str, t: torch.Tensor, index: int, dtype: torch.dtype, shape: tuple) -> int:
    """The address of a contiguous tensor of this device, type and shape."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        _fail(name, t, index, dtype, shape)
    return t.data_ptr()


def _rows(name: str, t: torch.Tensor, index: int, dtype: torch.dtype, shape: tuple) -> int:
    """The address of a tensor of this device, type and shape with inner stride 1."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape:
        _fail(name, t, index, dtype, shape)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: inner stride 1 is required")
    return t.data_ptr()


def _scalar(name: str, t: torch.Tensor, index: int, dtype: torch.dtype) -> int:
    if t.dtype is not dtype or t.get_device() != index or t.numel() != 1:
        raise ValueError(f"{name} must be a one-element {dtype} tensor on cuda:{index}")
    return t.data_ptr()


def _table(name: str, t: torch.Tensor, index: int, rows: int) -> Tuple[int, int, int]:
    """Address, row stride and columns of an int32 page table of so many rows (-1: any)."""
    if t.dtype is not _I32 or t.get_device() != index or t.dim() != 2 or (rows >= 0 and t.shape[0] != rows):
        raise ValueError(f"{name}: an int32 [{'?' if rows < 0 else rows}, pages] tensor on cuda:{index} is required, "
                         f"got {t.dtype} {list(t.shape)} on {t.device}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name}: inner stride 1 is required")
    return t.data_ptr(), t.stride(0), t.shape[1]


def _cache(cache: torch.Tensor, kv_scale: Optional[torch.Tensor]) -> Tuple[int, int, Optional[int]]:
    """Device index, format and scale address of a cache."""
    index = cache.get_device()
    if index < 0 or cache.dim() != 3 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous CUDA tensor [num_blocks, block_size, row]")
    row, dtype = cache.shape[2], cache.dtype
    if dtype is _U8 and row == E.MX_ROW:
        fmt = E.MLA_CACHE_MX
    elif dtype is _BF16 and row == E.ROW:
        fmt = E.MLA_CACHE_BF16
    elif dtype is _U8 and row == E.ROW:
        fmt = E.MLA_CACHE_E4M3
    else:
        raise ValueError("cache rows must be 576 bf16, 576 uint8 (e4m3) or 656 uint8 (microscaled)")
    if (kv_scale is not None) != (fmt == E.MLA_CACHE_E4M3):
        raise ValueError("kv_scale belongs to an e4m3 cache ([..., 576] uint8), and to no other")
    return index, fmt, None if kv_scale is None else _scalar("kv_scale", kv_scale, index, _F32)


def _stream(stream: Optional[torch.cuda.Stream], index: int) -> torch.cuda.Stream:
    if stream is None:
        return torch.cuda.current_stream(index)
    if stream.device_index != index:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to cuda:{index}")
    return stream


def _launch(index: int, what: str, entry, *args) -> None:
    """Calls a C entry point with the tensors' device current."""
    if torch.cuda.current_device() == index:
        rc = entry(*args)
    else:
        with torch.cuda.device(index):
            rc = entry(*args)
    if rc != E.MLA_OK:
        raise E.MlaError(rc, what)


def _empty(index: int, stream: Optional[torch.cuda.Stream], dtype: torch.dtype, *shape: int) -> torch.Tensor:
    """Uninitialised memory that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=index)  # (0.8 us less than with the shape as a tuple)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=index)


def mla_latent_cache_insert(
        kv_c: torch.Tensor, k_pe: torch.Tensor, cache: torch.Tensor, slot_mapping: torch.Tensor, *,
        norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
        positions: Optional[torch.Tensor] = None, cos_sin: Optional[torch.Tensor] = None,
        kv_scale: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
        pdl: bool = False, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Writes one latent row per token into ``cache`` (``mla_latent_insert_launch``).

    ``kv_c`` bf16 [T, 512] and ``k_pe`` bf16 [T, 64] (inner stride 1),
    ``slot_mapping`` int64 [T] (negative: no row).  With ``norm_weight`` (bf16
    [512]) the latents are RMS-normalised first; with ``cos_sin`` (fp32 [rows,
    64]) and ``positions`` (int32 [T]) the rotary values are rotated.  With
    ``pdl`` the previous kernel on the stream may write ``kv_c`` and ``k_pe``
    only: everything else is read while it may still be running.  A step that
    takes its query rows from the epilogue gives that a cache without pages
    (``torch.empty((0, block, 576))``) and slots of -1, in a call of its own.
    """
    index, fmt, scale = _cache(cache, kv_scale)
    T = kv_c.shape[0]
    x = _rows("kv_c", kv_c, index, _BF16, (T, E.NOPE))
    pe = _rows("k_pe", k_pe, index, _BF16, (T, E.PE))
    slots = _flat("slot_mapping", slot_mapping, index, _I64, (T,))
    w = None if norm_weight is None else _flat("norm_weight", norm_weight, index, _BF16, (E.NOPE,))
    flags, pos, tab, tab_rows = E.MLA_FLAG_PDL if pdl else 0, None, None, 0
    if cos_sin is not None or positions is not None:
        if cos_sin is None or positions is None:
            raise ValueError("rotation needs both positions and cos_sin")
        tab_rows = cos_sin.shape[0]
        tab = _flat("cos_sin", cos_sin, index, _F32, (tab_rows, E.PE))
        pos = _flat("positions", positions, index, _I32, (T,))
        flags |= E.MLA_FLAG_ROPE
    st = None if status is None else _scalar("status", status, index, _I32)
    _launch(index, "mla_latent_insert_launch", E.lib().mla_latent_insert_launch,
            x, kv_c.stride(0), pe, k_pe.stride(0), slots, w, eps, pos, tab, tab_rows, scale, T, cache.shape[1],
            cache.shape[0], fmt, flags, cache.data_ptr(), st, _stream(stream, index).cuda_stream)


def mla_latent_cache_gather(
        cache: torch.Tensor, block_table: torch.Tensor, cu_rows: torch.Tensor, rows: int, *,
        first: Optional[torch.Tensor] = None, kv_scale: Optional[torch.Tensor] = None,
        out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
        pdl: bool = False, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Rows of paged sequences as bf16 [rows, 576] (``mla_latent_gather_launch``).

    Sequence b's rows, from its position ``first[b]`` (0 without ``first``) on,
    land in ``out[cu_rows[b]:cu_rows[b+1]]``; ``block_table`` is int32 [B,
    pages], ``cu_rows`` int32 [B + 1], ascending.  Rows of ``out`` that belong
    to no sequence stay as they were (uninitialised in an ``out`` made here).
    With ``pdl`` everything is read after the previous kernel on the stream.
    """
    index, fmt, scale = _cache(cache, kv_scale)
    table, table_stride, cols = _table("block_table", block_table, index, -1)
    B = block_table.shape[0]
    cu = _flat("cu_rows", cu_rows, index, _I32, (B + 1,))
    at = None if first is None else _flat("first", first, index, _I32, (B,))
    st = None if status is None else _scalar("status", status, index, _I32)
    handle = _stream(stream, index).cuda_stream
    if out is None:
        if rows < 0:
            raise ValueError("rows must not be negative")
        out = _empty(index, stream, _BF16, rows, E.ROW)
        dst, dst_stride = out.data_ptr(), E.ROW
    else:
        dst, dst_stride = _rows("out", out, index, _BF16, (rows, E.ROW)), out.stride(0)
    _launch(index, "mla_latent_gather_launch", E.lib().mla_latent_gather_launch,
            cache.data_ptr(), fmt, cache.shape[1], cache.shape[0], scale, table, table_stride, cols, cu, at, B, rows,
            E.MLA_FLAG_PDL if pdl else 0, dst, dst_stride, st, handle)
    return out


_sm_counts = {}


def _sm_count(index: int) -> int:
    n = _sm_counts.get(index)
    if n is None:
        n = _sm_counts[index] = torch.cuda.get_device_properties(index).multi_processor_count
    return n


_workspace_bytes = functools.lru_cache(maxsize=256)(E.mla_prefix_attend_workspace_for)


def mla_prefix_decode_attention(
        q: torch.Tensor, cache: torch.Tensor, block_table: Optional[torch.Tensor],
        seq_lens: Optional[torch.Tensor], *, sm_scale: float,
        prefix_table: Optional[torch.Tensor] = None, prefix_lens: Optional[torch.Tensor] = None,
        group_offsets: Optional[torch.Tensor] = None,
        q_scale: Optional[torch.Tensor] = None, kv_scale: Optional[torch.Tensor] = None,
        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
        workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
        pdl: bool = False, stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Decode attention over the paged latent cache (``mla_prefix_attend_launch``);
    returns ``(out bf16 [T, H, 512], lse fp32 [T, H])``.

    ``q`` is [T, H, 576] bf16, or uint8 e4m3 bytes with ``q_scale``.  Token t
    attends to ``prefix_lens[g]`` keys of its group g and to ``seq_lens[t]``
    keys of its own pages ``block_table[t]`` (int32 [T, pages]; None: no keys
    of their own).  ``prefix_table`` is int32 [G, pages]; group g holds the
    tokens ``group_offsets[g] .. group_offsets[g + 1] - 1`` (int32 [G + 1]; None
    with one group: every token).  Without ``prefix_table`` there are no
    prefixes.  A ``workspace`` (uint8, at least ``mla_prefix_attend_workspace_for``
    bytes, or ``mla_prefix_attend_workspace`` for any cache) must not be shared by
    calls that may run at the same time; without one each call takes its own.
    Rows whose computation a timeout cut short (``MLA_STATUS_TIMEOUT`` in
    ``status``) are NaN.

    Where the cache needs decoding (or has odd pages) and groups have 256 rows
    (token, head) or more on average, the workspace has room for all of
    ``prefix_table``'s width, up to 73856 bytes for 64 keys; beyond 2 GiB there is
    none, and prefixes are decoded once for each 64 rows, which takes up to 1.8
    times as long.  So a table is best no wider than its longest prefix.
    """
    index, fmt, scale = _cache(cache, kv_scale)
    if q.dim() != 3:
        raise ValueError("q must be [T, H, 576]")
    T, H, _ = q.shape
    q_st, q_sh, _ = q.stride()
    blocks, block, _ = cache.shape
    flags = E.MLA_FLAG_PDL if pdl else 0
    if q_scale is None:
        qp, qs = _rows("q", q, index, _BF16, (T, H, E.ROW)), None
    else:
        qp, qs = _rows("q", q, index, _U8, (T, H, E.ROW)), _scalar("q_scale", q_scale, index, _F32)
        flags |= E.MLA_FLAG_Q_FP8
    table, table_stride, cols, lens = None, 0, 0, None
    if block_table is not None or seq_lens is not None:
        if block_table is None or seq_lens is None:
            raise ValueError("block_table and seq_lens go together")
        table, table_stride, cols = _table("block_table", block_table, index, T)
        lens = _flat("seq_lens", seq_lens, index, _I32, (T,))
    G, ptable, pstride, pcols, plens, offsets = 0, None, 0, 0, None, None
    if prefix_table is not None:
        if prefix_lens is None:
            raise ValueError("prefix_table and prefix_lens go together")
        ptable, pstride, pcols = _table("prefix_table", prefix_table, index, -1)
        G = prefix_table.shape[0]
        plens = _flat("prefix_lens", prefix_lens, index, _I32, (G,))
        if group_offsets is not None:
            offsets = _flat("group_offsets", group_offsets, index, _I32, (G + 1,))
    elif prefix_lens is not None or group_offsets is not None:
        raise ValueError("prefix_lens and group_offsets need prefix_table")
    st = None if status is None else _scalar("status", status, index, _I32)
    handle = _stream(stream, index).cuda_stream
    if out is None:
        out = _empty(index, stream, _BF16, T, H, E.NOPE)
        outp = out.data_ptr()
    else:
        outp = _flat("out", out, index, _BF16, (T, H, E.NOPE))
    if lse is None:
        lse = _empty(index, stream, _F32, T, H)
        lsep = lse.data_ptr()
    else:
        lsep = _flat("lse", lse, index, _F32, (T, H))
    if workspace is None:
        nbytes = _workspace_bytes(T, H, G, pcols * block, fmt, flags & E.MLA_FLAG_Q_FP8, block, blocks, _sm_count(index))
        workspace = _empty(index, stream, _U8, nbytes)
        ws = workspace.data_ptr()
    elif workspace.dim() != 1:
        raise ValueError("workspace must be a one-dimensional uint8 tensor")
    else:
        nbytes = workspace.numel()
        ws = _flat("workspace", workspace, index, _U8, (nbytes,))
    _launch(index, "mla_prefix_attend_launch", E.lib().mla_prefix_attend_launch,
            qp, q_st, q_sh, qs, cache.data_ptr(), fmt, block, blocks, scale,
            ptable, pstride, pcols, plens, offsets, G, table, table_stride, cols, lens, T, H, sm_scale, flags,
            outp, lsep, ws, nbytes, st, handle)
    return out, lse
