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

import torch

from . import MoEError, _check, lib

__all__ = ["attn_workspace_size", "alloc_attn_workspace", "rope_table", "rope_append", "attn_prefill",
           "attn_prefill_paged", "attn_decode"]

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


_P, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_HP, _CP = ctypes.POINTER(_Heads), ctypes.POINTER(_Cache)

SIGNATURES = {
    "moe_attn_workspace_size": (_SZ, [_I] * 5),
    "moe_rope_append": (_I, [_HP, _HP, _HP, _P, _P, _F, _P, _I, _I, _I, _P, _P, _I, _I, _I, _I, _I, _P, _CP,
                             _P, _SZ, _P]),
    "moe_attn_prefill": (_I, [_HP, _HP, _HP, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "moe_attn_prefill_paged": (_I, [_HP, _CP, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ,
                                    _P]),
    "moe_attn_decode": (_I, [_HP, _CP, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
}


def _tensor(t, name, dtype, dims, device=None):
    if not isinstance(t, torch.Tensor):
        raise MoEError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise MoEError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise MoEError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise MoEError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dims:
        raise MoEError(f"{name} must have {dims} dimensions, got {t.dim()}")


def _dense(t, name, dtype, shape, device):
    _tensor(t, name, dtype, len(shape), device)
    if tuple(t.shape) != tuple(shape):
        raise MoEError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise MoEError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(t, name, q=None):
    """A [tokens, heads, D] view: any token and head stride, dense D."""
    if q is None:
        if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
            raise MoEError(f"{name} must be a bfloat16 or float16 torch.Tensor")
        _tensor(t, name, t.dtype, 3)
        if t.get_device() != torch.cuda.current_device():
            raise MoEError(f"{name} must be on the current CUDA device")
    else:
        _tensor(t, name, q.dtype, 3, q.device)
        if t.shape[2] != q.shape[2]:
            raise MoEError(f"{name} must have head size {q.shape[2]}, got {t.shape[2]}")
    if t.stride(2) != 1 and t.shape[2] != 1 and t.numel() > 0:
        raise MoEError(f"{name} must be contiguous in its last dimension")
    return _Heads(t.data_ptr(), t.stride(0), t.stride(1))


def _cache(k_cache, v_cache, q):
    _tensor(k_cache, "k_cache", q.dtype, 4, q.device)
    pages, Hkv, page_size, D = k_cache.shape
    if D != q.shape[2]:
        raise MoEError(f"k_cache must have head size {q.shape[2]}, got {D}")
    if not k_cache.is_contiguous():
        raise MoEError("k_cache must be contiguous")
    _dense(v_cache, "v_cache", q.dtype, k_cache.shape, q.device)
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), pages, page_size), Hkv


def _launch_stream(stream, *made):
    """The stream to launch on; what this module allocated on the current
    stream stays reserved until the work on another one is done."""
    current = torch.cuda.current_stream()
    if stream is None or stream == current:
        return current.cuda_stream
    for t in made:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def attn_workspace_size(T: int, n_seq: int, Hq: int, Hkv: int, D: int) -> int:
    """Bytes of workspace of an attention call with up to T query rows and
    n_seq sequences (0 for an unsupported shape)."""
    return int(lib().moe_attn_workspace_size(T, n_seq, Hq, Hkv, D))


def alloc_attn_workspace(T: int, n_seq: int, Hq: int, Hkv: int, D: int, device="cuda") -> torch.Tensor:
    n = attn_workspace_size(T, n_seq, Hq, Hkv, D)
    if n == 0:
        raise MoEError("unsupported shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _workspace(workspace, T, n_seq, Hq, Hkv, D, device):
    """(tensor, whether it was made here)"""
    if workspace is None:
        return alloc_attn_workspace(T, n_seq, Hq, Hkv, D, device), True
    _tensor(workspace, "workspace", torch.uint8, 1, device)
    if not workspace.is_contiguous():
        raise MoEError("workspace must be contiguous")
    return workspace, False


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
    hq = _heads(q, "q")
    hk, hv = _heads(k, "k", q), _heads(v, "v", q)
    T, Hq, D = q.shape
    cache, Hkv = _cache(k_cache, v_cache, q)
    if tuple(k.shape) != (T, Hkv, D) or tuple(v.shape) != (T, Hkv, D):
        raise MoEError(f"k and v must have shape {(T, Hkv, D)}, got {tuple(k.shape)} and {tuple(v.shape)}")
    dev = q.device
    _tensor(table, "table", torch.float32, 2, dev)
    if not table.is_contiguous():
        raise MoEError("table must be contiguous")
    pos, slot = _dense(positions, "positions", torch.int32, (T,), dev), _dense(slots, "slots", torch.int32, (T,), dev)
    qn = None if q_norm is None else _dense(q_norm, "q_norm", torch.float32, (D,), dev)
    kn = None if k_norm is None else _dense(k_norm, "k_norm", torch.float32, (D,), dev)
    made = []
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=q.dtype, device=dev)
        made.append(q_out)
    out = _dense(q_out, "q_out", q.dtype, (T, Hq, D), dev)
    workspace, own = _workspace(workspace, max(T, 1), 0, Hq, Hkv, D, dev)
    if own:
        made.append(workspace)
    rc = lib().moe_rope_append(hq, hk, hv, qn, kn, eps, table.data_ptr(), table.shape[0], table.shape[1],
                               1 if interleaved else 0, pos, slot, T, Hq, Hkv, D, _DTYPES[q.dtype], out, cache,
                               workspace.data_ptr(), workspace.numel(), _launch_stream(stream, *made))
    _check(rc, "moe_rope_append")
    return q_out


def _results(q, out, lse, made):
    T, Hq, D = q.shape
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
        made.append(out)
    o = _dense(out, "out", q.dtype, (T, Hq, D), q.device)
    return out, o, None if lse is None else _dense(lse, "lse", torch.float32, (T, Hq), q.device)


def attn_prefill(q, k, v, q_starts, kv_starts, causal=True, scale=None, out=None, lse=None, workspace=None,
                 stream=None):
    """Attention of packed sequences: q [T, Hq, D], k and v [Tk, Hkv, D];
    sequence s has the rows q_starts[s] .. q_starts[s+1] and the keys
    kv_starts[s] .. kv_starts[s+1] (int32 [n_seq + 1]).  With ``causal`` the
    last row of a sequence sees its last key.  Returns out [T, Hq, D];
    ``lse`` (fp32 [T, Hq]) optionally receives the log of the softmax
    denominators.  ``scale`` defaults to 1 / sqrt(D)."""
    hq = _heads(q, "q")
    hk, hv = _heads(k, "k", q), _heads(v, "v", q)
    T, Hq, D = q.shape
    Tk, Hkv = k.shape[0], k.shape[1]
    if v.shape != k.shape:
        raise MoEError(f"v must have shape {tuple(k.shape)}, got {tuple(v.shape)}")
    _tensor(q_starts, "q_starts", torch.int32, 1, q.device)
    n = q_starts.shape[0] - 1
    if n < 0:
        raise MoEError("q_starts must have n_seq + 1 entries")
    qs = _dense(q_starts, "q_starts", torch.int32, (n + 1,), q.device)
    ks = _dense(kv_starts, "kv_starts", torch.int32, (n + 1,), q.device)
    made = []
    out, o, le = _results(q, out, lse, made)
    workspace, own = _workspace(workspace, max(T, 1), n, Hq, Hkv, D, q.device)
    if own:
        made.append(workspace)
    rc = lib().moe_attn_prefill(hq, hk, hv, qs, ks, n, T, Tk, Hq, Hkv, D, _DTYPES[q.dtype], 1 if causal else 0,
                                D ** -0.5 if scale is None else scale, o, le, workspace.data_ptr(),
                                workspace.numel(), _launch_stream(stream, *made))
    _check(rc, "moe_attn_prefill")
    return out


def _table(page_table, n, device):
    _tensor(page_table, "page_table", torch.int32, 2, device)
    return _dense(page_table, "page_table", torch.int32, (n, page_table.shape[1]), device), page_table.shape[1]


def attn_prefill_paged(q, k_cache, v_cache, page_table, q_starts, kv_lens, causal=True, scale=None, out=None,
                       lse=None, workspace=None, stream=None):
    """``attn_prefill`` with the keys in the paged cache: sequence s reads
    kv_lens[s] keys (int32 [n_seq]) on the pages page_table[s] (int32
    [n_seq, table_pages])."""
    hq = _heads(q, "q")
    T, Hq, D = q.shape
    cache, Hkv = _cache(k_cache, v_cache, q)
    _tensor(kv_lens, "kv_lens", torch.int32, 1, q.device)
    n = kv_lens.shape[0]
    lens = _dense(kv_lens, "kv_lens", torch.int32, (n,), q.device)
    qs = _dense(q_starts, "q_starts", torch.int32, (n + 1,), q.device)
    table, wide = _table(page_table, n, q.device)
    made = []
    out, o, le = _results(q, out, lse, made)
    workspace, own = _workspace(workspace, max(T, 1), n, Hq, Hkv, D, q.device)
    if own:
        made.append(workspace)
    rc = lib().moe_attn_prefill_paged(hq, cache, table, wide, qs, lens, n, T, Hq, Hkv, D, _DTYPES[q.dtype],
                                      1 if causal else 0, D ** -0.5 if scale is None else scale, o, le,
                                      workspace.data_ptr(), workspace.numel(), _launch_stream(stream, *made))
    _check(rc, "moe_attn_prefill_paged")
    return out


def attn_decode(q, k_cache, v_cache, page_table, kv_lens, prefix_table=None, prefix_len=0, scale=None, out=None,
                lse=None, workspace=None, stream=None):
    """Attention of one new token for each of B sequences: q [B, Hq, D].
    Row b sees the shared prefix (``prefix_len`` tokens on the pages
    ``prefix_table``, int32) and then its own kv_lens[b] tokens on the pages
    page_table[b]; the prefix is read once for the whole batch."""
    hq = _heads(q, "q")
    B, Hq, D = q.shape
    cache, Hkv = _cache(k_cache, v_cache, q)
    lens = _dense(kv_lens, "kv_lens", torch.int32, (B,), q.device)
    table, wide = _table(page_table, B, q.device)
    prefix = None
    if prefix_len > 0:
        if prefix_table is None:
            raise MoEError("prefix_len > 0 needs a prefix_table")
        prefix = _dense(prefix_table, "prefix_table", torch.int32, (prefix_table.numel(),), q.device)
        if prefix_table.numel() * cache.page_size < prefix_len:
            raise MoEError(f"prefix_table holds {prefix_table.numel()} pages, too few for {prefix_len} tokens")
    made = []
    out, o, le = _results(q, out, lse, made)
    workspace, own = _workspace(workspace, max(B, 1), B, Hq, Hkv, D, q.device)
    if own:
        made.append(workspace)
    rc = lib().moe_attn_decode(hq, cache, table, wide, lens, prefix, prefix_len, B, Hq, Hkv, D, _DTYPES[q.dtype],
                               D ** -0.5 if scale is None else scale, o, le, workspace.data_ptr(),
                               workspace.numel(), _launch_stream(stream, *made))
    _check(rc, "moe_attn_decode")
    return out
