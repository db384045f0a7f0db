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

from typing import Optional, Tuple

import torch

from . import epilogue as E


def _check(name: str, t: Optional[torch.Tensor], device: torch.device, dtype: torch.dtype, shape: tuple) -> None:
    """A tensor (if given) of this device, type and shape (None: any size)."""
    if t is None:
        return
    if t.device != device or t.dtype != dtype:
        raise ValueError(f"{name}: a {dtype} tensor on {device} is required, got {t.dtype} on {t.device}")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        want = ", ".join("?" if n is None else str(n) for n in shape)
        raise ValueError(f"{name}: shape [{want}] is required, got {list(t.shape)}")


def _flat(name: str, t: Optional[torch.Tensor]) -> None:
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _inner(name: str, t: torch.Tensor) -> None:
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: inner stride 1 is required")


def _scalar(name: str, t: Optional[torch.Tensor], device: torch.device) -> None:
    if t is not None and (t.dtype != torch.float32 or t.device != device or t.numel() != 1):
        raise ValueError(f"{name} must be a one-element fp32 tensor on {device}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _cache_format(cache: torch.Tensor, kv_scale: Optional[torch.Tensor]) -> int:
    if not cache.is_cuda or cache.dim() != 3 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous CUDA tensor [num_blocks, block_size, row]")
    if cache.dtype == torch.bfloat16 and cache.shape[2] == E.ROW:
        fmt = E.MLA_CACHE_BF16
    elif cache.dtype == torch.uint8 and cache.shape[2] == E.ROW:
        fmt = E.MLA_CACHE_E4M3
    elif cache.dtype == torch.uint8 and cache.shape[2] == E.MX_ROW:
        fmt = E.MLA_CACHE_MX
    else:
        raise ValueError("cache rows must be 576 bf16, 576 uint8 (e4m3) or 656 uint8 (microscaled)")
    if (kv_scale is not None) != (fmt == E.MLA_CACHE_E4M3):
        raise ValueError("kv_scale belongs to an e4m3 cache ([..., 576] uint8), and to no other")
    _scalar("kv_scale", kv_scale, cache.device)
    return fmt


def _status(status: Optional[torch.Tensor], device: torch.device) -> None:
    if status is not None and (status.dtype != torch.int32 or status.device != device or status.numel() != 1):
        raise ValueError(f"status must be a one-element int32 tensor on {device}")


def _stream(stream: Optional[torch.cuda.Stream], device: torch.device) -> torch.cuda.Stream:
    if stream is None:
        return torch.cuda.current_stream(device)
    if stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    return stream


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
    64]) and ``positions`` (int32 [T]) the rotary values are rotated.
    """
    device = cache.device
    fmt = _cache_format(cache, kv_scale)
    T = kv_c.shape[0]
    _check("kv_c", kv_c, device, torch.bfloat16, (T, E.NOPE))
    _check("k_pe", k_pe, device, torch.bfloat16, (T, E.PE))
    _check("slot_mapping", slot_mapping, device, torch.int64, (T,))
    _check("norm_weight", norm_weight, device, torch.bfloat16, (E.NOPE,))
    _inner("kv_c", kv_c)
    _inner("k_pe", k_pe)
    _flat("slot_mapping", slot_mapping)
    _flat("norm_weight", norm_weight)
    if (cos_sin is None) != (positions is None):
        raise ValueError("rotation needs both positions and cos_sin")
    _check("positions", positions, device, torch.int32, (T,))
    _check("cos_sin", cos_sin, device, torch.float32, (None, E.PE))
    _flat("positions", positions)
    _flat("cos_sin", cos_sin)
    _status(status, device)
    flags = (E.MLA_FLAG_ROPE if cos_sin is not None else 0) | (E.MLA_FLAG_PDL if pdl else 0)
    s = _stream(stream, device)
    with torch.cuda.device(device):
        rc = E.mla_latent_insert_launch(
            _ptr(kv_c), kv_c.stride(0), _ptr(k_pe), k_pe.stride(0), _ptr(slot_mapping), _ptr(norm_weight), eps,
            _ptr(positions), _ptr(cos_sin), 0 if cos_sin is None else cos_sin.shape[0], _ptr(kv_scale),
            T, cache.shape[1], cache.shape[0], fmt, flags, _ptr(cache), _ptr(status), s.cuda_stream)
    if rc != E.MLA_OK:
        raise E.MlaError(rc, "mla_latent_insert_launch")


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
    """
    device = cache.device
    fmt = _cache_format(cache, kv_scale)
    _check("block_table", block_table, device, torch.int32, (None, None))
    _inner("block_table", block_table)
    B = block_table.shape[0]
    _check("cu_rows", cu_rows, device, torch.int32, (B + 1,))
    _check("first", first, device, torch.int32, (B,))
    _flat("cu_rows", cu_rows)
    _flat("first", first)
    _status(status, device)
    s = _stream(stream, device)
    if out is None:
        with torch.cuda.stream(s):
            out = torch.empty((rows, E.ROW), dtype=torch.bfloat16, device=device)
    else:
        _check("out", out, device, torch.bfloat16, (rows, E.ROW))
        _inner("out", out)
    with torch.cuda.device(device):
        rc = E.mla_latent_gather_launch(
            _ptr(cache), fmt, cache.shape[1], cache.shape[0], _ptr(kv_scale), _ptr(block_table),
            block_table.stride(0), block_table.shape[1], _ptr(cu_rows), _ptr(first), B, rows,
            E.MLA_FLAG_PDL if pdl else 0, _ptr(out), out.stride(0), _ptr(status), s.cuda_stream)
    if rc != E.MLA_OK:
        raise E.MlaError(rc, "mla_latent_gather_launch")
    return out


_sm_counts = {}


def _sm_count(device: torch.device) -> int:
    n = _sm_counts.get(device.index)
    if n is None:
        n = _sm_counts[device.index] = torch.cuda.get_device_properties(device).multi_processor_count
    return n


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
    prefixes.  A ``workspace`` (uint8, at least ``mla_prefix_attend_workspace``
    bytes) must not be shared by calls that may run at the same time; without
    one each call takes its own.
    """
    device = cache.device
    fmt = _cache_format(cache, kv_scale)
    if q.dim() != 3:
        raise ValueError("q must be [T, H, 576]")
    T, H = q.shape[0], q.shape[1]
    _check("q", q, device, torch.bfloat16 if q_scale is None else torch.uint8, (T, H, E.ROW))
    _inner("q", q)
    _scalar("q_scale", q_scale, device)
    if (block_table is None) != (seq_lens is None):
        raise ValueError("block_table and seq_lens go together")
    _check("block_table", block_table, device, torch.int32, (T, None))
    _check("seq_lens", seq_lens, device, torch.int32, (T,))
    _flat("seq_lens", seq_lens)
    G = 0
    if (prefix_table is None) != (prefix_lens is None) or (prefix_table is None and group_offsets is not None):
        raise ValueError("prefix_table and prefix_lens go together, group_offsets with them")
    if prefix_table is not None:
        G = prefix_table.shape[0]
        _check("prefix_table", prefix_table, device, torch.int32, (None, None))
        _check("prefix_lens", prefix_lens, device, torch.int32, (G,))
        _check("group_offsets", group_offsets, device, torch.int32, (G + 1,))
        _inner("prefix_table", prefix_table)
        _flat("prefix_lens", prefix_lens)
        _flat("group_offsets", group_offsets)
    if block_table is not None:
        _inner("block_table", block_table)
    _status(status, device)
    s = _stream(stream, device)
    with torch.cuda.device(device), torch.cuda.stream(s):
        if out is None:
            out = torch.empty((T, H, E.NOPE), dtype=torch.bfloat16, device=device)
        else:
            _check("out", out, device, torch.bfloat16, (T, H, E.NOPE))
            _flat("out", out)
        if lse is None:
            lse = torch.empty((T, H), dtype=torch.float32, device=device)
        else:
            _check("lse", lse, device, torch.float32, (T, H))
            _flat("lse", lse)
        if workspace is None:
            need = E.mla_prefix_attend_workspace(T, H, G, _sm_count(device))
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            _check("workspace", workspace, device, torch.uint8, (None,))
            _flat("workspace", workspace)
        rc = E.mla_prefix_attend_launch(
            _ptr(q), q.stride(0), q.stride(1), _ptr(q_scale), _ptr(cache), fmt, cache.shape[1], cache.shape[0],
            _ptr(kv_scale), _ptr(prefix_table), 0 if G == 0 else prefix_table.stride(0),
            0 if G == 0 else prefix_table.shape[1], _ptr(prefix_lens), _ptr(group_offsets), G,
            _ptr(block_table), 0 if block_table is None else block_table.stride(0),
            0 if block_table is None else block_table.shape[1], _ptr(seq_lens), T, H, sm_scale,
            (E.MLA_FLAG_Q_FP8 if q_scale is not None else 0) | (E.MLA_FLAG_PDL if pdl else 0),
            _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(status), s.cuda_stream)
    if rc != E.MLA_OK:
        raise E.MlaError(rc, "mla_prefix_attend_launch")
    return out, lse
