"""Attention of the decoder layer the MoE layer belongs to: the binding of the
``moe_rope_append`` / ``moe_attn_*`` entry points (``include/moe.h``).

``rope_append`` norms and rotates a projection's queries and keys and appends
keys and values to a paged cache; ``attn_prefill`` / ``attn_prefill_paged``
attend over whole prompts, ``attn_decode`` over the cache for one new token
of each sequence, with an optional prefix that the whole batch shares.  As in
the rest of the package the functions only check and marshal arguments.

A cache is two tensors [pages, Hkv, page_size, D]; a page table row lists a
sequence's pages, token j sits in row j % page_size of page j // page_size.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import MoEError, _check, lib

__all__ = ["attn_workspace_size", "alloc_attn_workspace", "rope_table", "rope_append", "attn_prefill",
           "attn_prefill_paged", "attn_decode"]

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8

# A call of a few microseconds on the GPU is bound by this module's host time:
# a tensor costs a handful of attribute reads (each about 0.1 us), the argument
# structs are packed as bytes, and the stream is read without wrapping it.
_HEADS = struct.Struct("=Qqq").pack      # moe_heads: data, token_stride, head_stride
_CACHE = struct.Struct("=QQii").pack     # moe_kv_cache: k, v, pages, page_size

_P, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

SIGNATURES = {
    "moe_attn_workspace_size": (_SZ, [_I] * 5),
    "moe_rope_append": (_I, [_P, _P, _P, _P, _P, _F, _P, _I, _I, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ,
                             _P]),
    "moe_attn_prefill": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "moe_attn_prefill_paged": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "moe_attn_decode": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
}


def _refuse(t, name, dtype, dims, device):
    """The reason why _dense or _view did not take a tensor."""
    if not isinstance(t, torch.Tensor):
        raise MoEError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise MoEError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise MoEError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.dtype != dtype:
        raise MoEError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(dims):
        raise MoEError(f"{name} must have {len(dims)} dimensions, got {t.dim()}")
    if any(want is not None and want != got for want, got in zip(dims, t.shape)):
        raise MoEError(f"{name} must have shape {tuple(dims)}, got {tuple(t.shape)}")
    raise MoEError(f"{name} must be contiguous")


def _dense(t, name, dtype, shape, device):
    """Address of a contiguous tensor of this type, shape (a tuple) and device."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _refuse(t, name, dtype, shape, device)


def _query(q):
    """(packed view, T, Hq, D, dtype, its code, device) of the queries [T, Hq, D]."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise MoEError("q must be a bfloat16 or float16 torch.Tensor")
    dtype = q.dtype
    device = torch.cuda.current_device() if q.is_cuda else -1
    if q.dim() != 3 or q.get_device() != device or device < 0:
        _refuse(q, "q", dtype, (None, None, None), device)
    T, Hq, D = q.shape
    st, sh, sd = q.stride()
    if sd != 1 and D > 1 and T * Hq > 0:
        raise MoEError("q must be contiguous in its last dimension")
    return _HEADS(q.data_ptr(), st, sh), T, Hq, D, dtype, _DTYPES[dtype], device


def _view(t, name, dtype, shape, device):
    """Packed [tokens, heads, D] view: any token and head stride, dense D."""
    try:
        ok = t.dtype is dtype and t.shape == shape and t.get_device() == device
    except AttributeError:
        ok = False
    if not ok:
        _refuse(t, name, dtype, shape, device)
    st, sh, sd = t.stride()
    if sd != 1 and shape[2] > 1 and shape[0] * shape[1] > 0:
        raise MoEError(f"{name} must be contiguous in its last dimension")
    return _HEADS(t.data_ptr(), st, sh)


def _cache(k_cache, v_cache, D, dtype, device):
    """(packed cache, Hkv, page_size)"""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4 or k_cache.shape[3] != D:
        _refuse(k_cache, "k_cache", dtype, (None, None, None, D), device)
    shape = k_cache.shape
    k = _dense(k_cache, "k_cache", dtype, shape, device)
    v = _dense(v_cache, "v_cache", dtype, shape, device)
    return _CACHE(k, v, min(shape[0], 0x7fffffff), shape[2]), shape[1], shape[2]


def _launch_stream(stream, device, made):
    """The stream to launch on; what was allocated here on the current stream
    stays reserved until the work on another one is done."""
    current = _raw_stream(device)
    if stream is None or stream.cuda_stream == current:
        return current
    for t in made:
        t.record_stream(stream)
    return stream.cuda_stream


def _raw_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    _raw_stream = torch._C._cuda_getCurrentRawStream  # noqa: F811  (the same value, without a Stream object)


def attn_workspace_size(T: int, n_seq: int, Hq: int, Hkv: int, D: int) -> int:
    """Bytes of workspace of an attention call with up to T query rows and
    n_seq sequences (0 for an unsupported shape)."""
    return int(lib().moe_attn_workspace_size(T, n_seq, Hq, Hkv, D))


def alloc_attn_workspace(T: int, n_seq: int, Hq: int, Hkv: int, D: int, device="cuda") -> torch.Tensor:
    n = attn_workspace_size(T, n_seq, Hq, Hkv, D)
    if n == 0:
        raise MoEError("unsupported shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _workspace(workspace, T, n_seq, Hq, Hkv, D, device, made):
    """(address, bytes)"""
    if workspace is None:
        workspace = alloc_attn_workspace(T, n_seq, Hq, Hkv, D, torch.device("cuda", device))
        made.append(workspace)
    n = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
    return _dense(workspace, "workspace", _U8, (n,), device), n


def rope_table(max_pos: int, rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               original_max_pos: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
               device="cuda") -> torch.Tensor:
    """The cos | sin table [max_pos, rot] fp32 that ``rope_append`` takes,
    built once when a model is loaded (angles in fp64).

    Angle i of position p is p * f_i, f_i = base^(-2i/rot).  ``scaling`` for
    contexts ``factor`` times longer than the trained ``original_max_pos``:
    "linear" divides every f_i by ``factor``; "by_parts" keeps frequencies
    that turn at least ``beta_fast`` times over the trained length, divides
    those that turn at most ``beta_slow`` times, blends linearly in i between
    the two, and scales cos and sin by 0.1 ln(factor) + 1 (so that attention
    logits grow by its square)."""
    if rot <= 0 or rot % 2 or max_pos <= 0 or not base > 1.0 or not factor >= 1.0:
        raise MoEError("rope_table: rot must be even and positive, max_pos positive, base > 1, factor >= 1")
    i = torch.arange(rot // 2, dtype=torch.float64)
    freq = base ** (-2.0 * i / rot)
    mul = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if not original_max_pos or original_max_pos <= 0:
            raise MoEError("rope_table: by_parts scaling needs original_max_pos")
        # index whose frequency turns `n` times over the trained length
        at = [rot * math.log(original_max_pos / (n * 2 * math.pi)) / (2 * math.log(base))
              for n in (beta_fast, beta_slow)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        keep = 1.0 - ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
        mul = 0.1 * math.log(factor) + 1.0
    elif scaling is not None:
        raise MoEError(f"rope_table: unknown scaling {scaling!r}")
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq.to(device)[None, :]
    return torch.cat([angle.cos() * mul, angle.sin() * mul], dim=1).float().contiguous()


def rope_append(q, k, v, table, positions, slots, k_cache, v_cache, q_norm=None, k_norm=None, eps=1e-6,
                interleaved=False, q_out=None, workspace=None, stream=None):
    """Norm (per head, optional) and rotate q [T, Hq, D] and k [T, Hkv, D],
    and write k and v [T, Hkv, D] to the paged cache; returns q_out.

    q, k, v may be strided views of one projection's rows.  ``table``
    [max_pos, rot] fp32 from ``rope_table``; ``positions`` and ``slots`` int32
    [T]; a slot is page * page_size + row, negative to leave the cache alone.
    ``q_norm`` / ``k_norm``: fp32 [D] weights or None."""
    hq, T, Hq, D, dtype, code, dev = _query(q)
    cache, Hkv, _ = _cache(k_cache, v_cache, D, dtype, dev)
    kv = (T, Hkv, D)
    hk, hv = _view(k, "k", dtype, kv, dev), _view(v, "v", dtype, kv, dev)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        _refuse(table, "table", _F32, (None, None), dev)
    max_pos, rot = table.shape
    tab = _dense(table, "table", _F32, (max_pos, rot), dev)
    pos, slot = _dense(positions, "positions", _I32, (T,), dev), _dense(slots, "slots", _I32, (T,), dev)
    qn = None if q_norm is None else _dense(q_norm, "q_norm", _F32, (D,), dev)
    kn = None if k_norm is None else _dense(k_norm, "k_norm", _F32, (D,), dev)
    made = []
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=dtype, device=q.device)
        made.append(q_out)
    out = _dense(q_out, "q_out", dtype, (T, Hq, D), dev)
    ws, n = _workspace(workspace, T or 1, 0, Hq, Hkv, D, dev, made)
    rc = lib().moe_rope_append(hq, hk, hv, qn, kn, eps, tab, max_pos, rot, 1 if interleaved else 0, pos, slot, T, Hq,
                               Hkv, D, code, out, cache, ws, n, _launch_stream(stream, dev, made))
    if rc:
        _check(rc, "moe_rope_append")
    return q_out


def _results(q, T, Hq, D, dtype, dev, out, lse, made):
    if out is None:
        out = torch.empty((T, Hq, D), dtype=dtype, device=q.device)
        made.append(out)
    return (out, _dense(out, "out", dtype, (T, Hq, D), dev),
            None if lse is None else _dense(lse, "lse", _F32, (T, Hq), dev))


def _entries(t, name, dev):
    """Entries of a one-dimensional int32 array."""
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        _refuse(t, name, _I32, (None,), dev)
    return t.shape[0]


def _page_table(t, n, dev):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        _refuse(t, "page_table", _I32, (n, None), dev)
    wide = t.shape[1]
    return _dense(t, "page_table", _I32, (n, wide), dev), wide


def attn_prefill(q, k, v, q_starts, kv_starts, causal=True, scale=None, out=None, lse=None, workspace=None,
                 stream=None):
    """Attention of packed sequences: q [T, Hq, D], k and v [Tk, Hkv, D];
    sequence s has the rows q_starts[s] .. q_starts[s+1] and the keys
    kv_starts[s] .. kv_starts[s+1] (int32 [n_seq + 1]).  With ``causal`` the
    last row of a sequence sees its last key.  Returns out [T, Hq, D];
    ``lse`` (fp32 [T, Hq]) optionally receives the log of the softmax
    denominators.  ``scale`` defaults to 1 / sqrt(D)."""
    hq, T, Hq, D, dtype, code, dev = _query(q)
    if not isinstance(k, torch.Tensor) or k.dim() != 3 or k.shape[2] != D:
        _refuse(k, "k", dtype, (None, None, D), dev)
    Tk, Hkv, _ = kv = tuple(k.shape)
    hk, hv = _view(k, "k", dtype, kv, dev), _view(v, "v", dtype, kv, dev)
    n = _entries(q_starts, "q_starts", dev) - 1
    if n < 0:
        raise MoEError("q_starts must have n_seq + 1 entries")
    qs, ks = _dense(q_starts, "q_starts", _I32, (n + 1,), dev), _dense(kv_starts, "kv_starts", _I32, (n + 1,), dev)
    made = []
    out, o, le = _results(q, T, Hq, D, dtype, dev, out, lse, made)
    ws, size = _workspace(workspace, T or 1, n, Hq, Hkv, D, dev, made)
    rc = lib().moe_attn_prefill(hq, hk, hv, qs, ks, n, T, Tk, Hq, Hkv, D, code, 1 if causal else 0,
                                D ** -0.5 if scale is None else scale, o, le, ws, size,
                                _launch_stream(stream, dev, made))
    if rc:
        _check(rc, "moe_attn_prefill")
    return out


def attn_prefill_paged(q, k_cache, v_cache, page_table, q_starts, kv_lens, causal=True, scale=None, out=None,
                       lse=None, workspace=None, stream=None):
    """``attn_prefill`` with the keys in the paged cache: sequence s reads
    kv_lens[s] keys (int32 [n_seq]) on the pages page_table[s] (int32
    [n_seq, table_pages])."""
    hq, T, Hq, D, dtype, code, dev = _query(q)
    cache, Hkv, _ = _cache(k_cache, v_cache, D, dtype, dev)
    n = _entries(kv_lens, "kv_lens", dev)
    lens, qs = _dense(kv_lens, "kv_lens", _I32, (n,), dev), _dense(q_starts, "q_starts", _I32, (n + 1,), dev)
    table, wide = _page_table(page_table, n, dev)
    made = []
    out, o, le = _results(q, T, Hq, D, dtype, dev, out, lse, made)
    ws, size = _workspace(workspace, T or 1, n, Hq, Hkv, D, dev, made)
    rc = lib().moe_attn_prefill_paged(hq, cache, table, wide, qs, lens, n, T, Hq, Hkv, D, code, 1 if causal else 0,
                                      D ** -0.5 if scale is None else scale, o, le, ws, size,
                                      _launch_stream(stream, dev, made))
    if rc:
        _check(rc, "moe_attn_prefill_paged")
    return out


def attn_decode(q, k_cache, v_cache, page_table, kv_lens, prefix_table=None, prefix_len=0, scale=None, out=None,
                lse=None, workspace=None, stream=None):
    """Attention of one new token for each of B sequences: q [B, Hq, D].
    Row b sees the shared prefix (``prefix_len`` tokens on the pages
    ``prefix_table``, int32) and then its own kv_lens[b] tokens on the pages
    page_table[b]; the prefix is read once for the whole batch."""
    hq, B, Hq, D, dtype, code, dev = _query(q)
    cache, Hkv, page_size = _cache(k_cache, v_cache, D, dtype, dev)
    lens = _dense(kv_lens, "kv_lens", _I32, (B,), dev)
    table, wide = _page_table(page_table, B, dev)
    prefix = None
    if prefix_len > 0:
        if prefix_table is None:
            raise MoEError("prefix_len > 0 needs a prefix_table")
        held = _entries(prefix_table, "prefix_table", dev)
        prefix = _dense(prefix_table, "prefix_table", _I32, (held,), dev)
        if held * page_size < prefix_len:
            raise MoEError(f"prefix_table holds {held} pages, too few for {prefix_len} tokens")
    made = []
    out, o, le = _results(q, B, Hq, D, dtype, dev, out, lse, made)
    ws, size = _workspace(workspace, B or 1, B, Hq, Hkv, D, dev, made)
    rc = lib().moe_attn_decode(hq, cache, table, wide, lens, prefix, prefix_len, B, Hq, Hkv, D, code,
                               D ** -0.5 if scale is None else scale, o, le, ws, size,
                               _launch_stream(stream, dev, made))
    if rc:
        _check(rc, "moe_attn_decode")
    return out
