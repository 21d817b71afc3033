"""Attention of the decoder layer the MoE layer belongs to: the binding of the
``moe_rope_append`` / ``moe_attn_*`` entry points (``include/moe.h``).

``rope_append`` norms and rotates a projection's queries and keys and appends
keys and values to a paged cache; ``attn_prefill`` / ``attn_prefill_paged``
attend over whole prompts, ``attn_decode`` over the cache for one new token
of each sequence, with an optional prefix that the whole batch shares.  As in
the rest of the package the functions only check and marshal arguments; here
they do so in compiled code (``_attn_binding.so``, 3 to 7 us a call instead of
11 to 17 through ctypes), which takes their places at the first call.

A cache is two tensors [pages, Hkv, page_size, D]; a page table row lists a
sequence's pages, token j sits in row j % page_size of page j // page_size.

``stream``: the stream to launch on (default: the current one).  Outputs and
workspaces that a call makes come from its memory; that the tensors passed in
are ready there, and kept until it is past them, is the caller's business, as
with any use of a tensor on another stream.
"""
from __future__ import annotations

import ctypes
import importlib
import inspect
import math
import sys

import torch

from . import MoEError, lib

__all__ = ["attn_workspace_size", "alloc_attn_workspace", "rope_table", "rope_append", "attn_prefill",
           "attn_prefill_paged", "attn_decode"]

_P, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

SIGNATURES = {
    "moe_attn_workspace_size": (_SZ, [_I] * 5),
    "moe_debug_attn_wait_timeout": (_I, [_I]),
    "moe_rope_append": (_I, [_P, _P, _P, _P, _P, _F, _P, _I, _I, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ,
                             _P]),
    "moe_attn_prefill": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "moe_attn_prefill_paged": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "moe_attn_decode": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
}

_native = None


def _load():
    """The compiled binding (csrc/attn_binding.cpp), connected to the library.

    Its functions take their parameters, defaults and documentation from the
    ones below and their place, in this module and in the package, on the first
    call; a name imported from here before that goes on through the one below
    (0.15 us more a call)."""
    global _native
    if _native is None:
        handle = lib()
        try:
            native = importlib.import_module("._attn_binding", __package__)
        except ImportError as e:
            raise MoEError("the attention binding is missing or does not load: build it with "
                           f"`python -m expert_layer_gb300._build` ({e})") from e
        native.bind(MoEError, *(ctypes.cast(getattr(handle, n), _P).value for n in (
            "moe_attn_workspace_size", "moe_rope_append", "moe_attn_prefill", "moe_attn_prefill_paged",
            "moe_attn_decode", "moe_error_string")), *(
                (tuple(inspect.signature(f).parameters), f.__defaults__ or (),
                 f"{f.__name__}{inspect.signature(f)}\n--\n\n{inspect.getdoc(f)}") for f in _FUNCTIONS))
        for name in (f.__name__ for f in _FUNCTIONS):
            for module in (sys.modules[__name__], sys.modules[__package__]):
                setattr(module, name, getattr(native, name))
        _native = native
    return _native


def attn_workspace_size(T: int, n_seq: int, Hq: int, Hkv: int, D: int) -> int:
    """Bytes of workspace of an attention call with up to T query rows and
    n_seq sequences (0 for an unsupported shape)."""
    return int(lib().moe_attn_workspace_size(T, n_seq, Hq, Hkv, D))


def alloc_attn_workspace(T: int, n_seq: int, Hq: int, Hkv: int, D: int, device="cuda") -> torch.Tensor:
    n = attn_workspace_size(T, n_seq, Hq, Hkv, D)
    if n == 0:
        raise MoEError("unsupported shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


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
    return _load().rope_append(q, k, v, table, positions, slots, k_cache, v_cache, q_norm, k_norm, eps, interleaved,
                               q_out, workspace, stream)


def attn_prefill(q, k, v, q_starts, kv_starts, causal=True, scale=None, out=None, lse=None, workspace=None,
                 stream=None):
    """Attention of packed sequences: q [T, Hq, D], k and v [Tk, Hkv, D];
    sequence s has the rows q_starts[s] .. q_starts[s+1] and the keys
    kv_starts[s] .. kv_starts[s+1] (int32 [n_seq + 1]).  q_starts go from 0 to
    T: rows outside are left as they were and reported (``read_status``);
    padding rows can be a last sequence without keys.  With ``causal`` the
    last row of a sequence sees its last key, and the values that a row does
    not see must be finite (a weight of 0 does not silence them).  Returns out [T, Hq, D];
    ``lse`` (fp32 [T, Hq]) optionally receives the log of the softmax
    denominators.  ``scale`` defaults to 1 / sqrt(D)."""
    return _load().attn_prefill(q, k, v, q_starts, kv_starts, causal, scale, out, lse, workspace, stream)


def attn_prefill_paged(q, k_cache, v_cache, page_table, q_starts, kv_lens, causal=True, scale=None, out=None,
                       lse=None, workspace=None, stream=None):
    """``attn_prefill`` with the keys in the paged cache: sequence s reads
    kv_lens[s] keys (int32 [n_seq]) on the pages page_table[s] (int32
    [n_seq, table_pages])."""
    return _load().attn_prefill_paged(q, k_cache, v_cache, page_table, q_starts, kv_lens, causal, scale, out, lse,
                                      workspace, stream)


def attn_decode(q, k_cache, v_cache, page_table, kv_lens, prefix_table=None, prefix_len=0, scale=None, out=None,
                lse=None, workspace=None, stream=None):
    """Attention of one new token for each of B sequences: q [B, Hq, D].
    Row b sees the shared prefix (``prefix_len`` tokens on the pages
    ``prefix_table``, int32) and then its own kv_lens[b] tokens on the pages
    page_table[b]; the prefix is read once for the whole batch."""
    return _load().attn_decode(q, k_cache, v_cache, page_table, kv_lens, prefix_table, prefix_len, scale, out, lse,
                               workspace, stream)


_FUNCTIONS = (rope_append, attn_prefill, attn_prefill_paged, attn_decode)
