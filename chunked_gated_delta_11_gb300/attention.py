"""Softmax attention beside the KDA layers: the binding of kda_attn_fwd,
kda_cache_append, kda_cache_attn, kda_cache_evict, kda_cache_reserve and
kda_cache_release (include/kda.h).

A hybrid model puts an attention layer after every few KDA layers.  It works on
the same packed rows ([T_total, H, 128] bf16, cu_seqlens), keeps its keys and
values in a paged cache of e4m3 codes with one scale per (page, KV head), and
can drop the cached tokens that got the least attention.  The pages of the cache
are taken from a pool, and given back, on the device.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
from typing import NamedTuple, Optional

import torch

from . import build as _build

MASKS = {"full": 0, "causal": 1, "prefix": 2}
PAGE_SIZES = (16, 32, 64, 128)


class KvCache(NamedTuple):
    """A pool of cache pages (kda_cache of include/kda.h); the tensors are the caller's."""
    k: torch.Tensor        # float8_e4m3fn [pages, Hk, page_size, 128]
    v: torch.Tensor        # float8_e4m3fn [pages, Hk, page_size, 128]
    k_scale: torch.Tensor  # float32 [pages, Hk]
    v_scale: torch.Tensor  # float32 [pages, Hk]
    pos: torch.Tensor      # int32 [pages, Hk, page_size]
    weight: torch.Tensor   # float32 [pages, Hk, page_size]


class Reservation(NamedTuple):
    """What kda_cache_reserve gives."""
    lens: torch.Tensor             # int32 [N], with the new rows (the old length where refused)
    cu_seqlens: torch.Tensor       # int32 [N + 1], packing of the new rows
    slots: Optional[torch.Tensor]  # int64 [rows], cache slot of every new row, -1 without one
    free_count: torch.Tensor       # int32 [1], pages left


class _AttnOptions(ctypes.Structure):
    _fields_ = [("mask", ctypes.c_int32), ("cap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("Hk", ctypes.c_int32), ("D", ctypes.c_int32)]


class _CacheAttnOptions(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("accumulate", ctypes.c_int32)]


def declare(lib):
    """Argument types of the entry points of this module."""
    P, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                            ctypes.c_size_t)
    lib.kda_attn_fwd.argtypes = [P, P, P, P, f32, P, i64, i32, i32, i32, i32, P, P]
    lib.kda_attn_fwd.restype = ctypes.c_int
    lib.kda_cache_append.argtypes = [P, P, P, P, i32, P, P, P, i64, i32, P]
    lib.kda_cache_append.restype = ctypes.c_int
    lib.kda_cache_attn_workspace_size.argtypes = [P, i64, i32, i32, i32, i32]
    lib.kda_cache_attn_workspace_size.restype = sz
    lib.kda_cache_attn.argtypes = [P, P, P, f32, P, i32, P, P, i64, i32, i32, P, P, sz, P]
    lib.kda_cache_attn.restype = ctypes.c_int
    lib.kda_cache_evict_workspace_size.argtypes = [P, i32, i32]
    lib.kda_cache_evict_workspace_size.restype = sz
    lib.kda_cache_evict.argtypes = [P, P, i32, P, P, i32, i32, i32, i32, P, P, sz, P]
    lib.kda_cache_evict.restype = ctypes.c_int
    lib.kda_cache_reserve.argtypes = [P, i32, P, P, P, P, i32, i32, i64, i32, P, P, P, P, P]
    lib.kda_cache_reserve.restype = ctypes.c_int
    lib.kda_cache_release.argtypes = [P, i32, P, P, P, P, i32, i32, i32, P, P]
    lib.kda_cache_release.restype = ctypes.c_int


_binding = None


def load_binding():
    """The extension that checks the tensors and calls libkda (built by build.py)."""
    global _binding
    if _binding is None:
        from . import load
        load()  # says so if libkda is not built
        was, now = _build.binding_built_for(), _build.binding_tag()
        if was != now:
            state = f"was built for {was}, this is {now}" if was else f"is not built ({_build.BINDING} missing)"
            raise RuntimeError(f"the attention binding {state}; run chunked_gated_delta_11_gb300.build.build()")
        loader = importlib.machinery.ExtensionFileLoader("attn_binding", _build.BINDING)
        spec = importlib.util.spec_from_file_location("attn_binding", _build.BINDING, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        _binding = module
    return _binding


def _run(stream, where, call, *args):
    """One call of the extension, on torch's current stream or on `stream` (where its
    outputs and workspace are then allocated too); raises on a status of libkda."""
    if stream is None:
        r = call(*args)
    else:
        with torch.cuda.stream(stream):
            r = call(*args)
    if type(r) is int and r != 0:
        from . import KdaError
        raise KdaError(r, where)
    return r


def kda_attn_fwd(q, k, v, scale, mask="causal", cap=0.0, slopes=None, prefix_lens=None,
                 cu_seqlens=None, N=None, out=None, stream=None):
    """Attention over packed rows: q [T_total, H, 128], k and v [T_total, Hk, 128]
    bf16.  mask: "causal", "full", or "prefix" (the first prefix_lens[n] rows of
    sequence n are seen by all of it); cap: scores become cap * tanh(x / cap);
    slopes: fp32 [H], subtracts slopes[h] * distance.  Returns out [T_total, H, 128]."""
    code = MASKS.get(mask)
    if code is None:
        raise ValueError(f"mask must be one of {tuple(MASKS)}, got {mask!r}")
    b = _binding or load_binding()
    return _run(stream, "kda_attn_fwd", b.attn_fwd, q, k, v, scale, code, cap, slopes, prefix_lens,
                cu_seqlens, N, out)


def kda_cache_alloc(pages, Hk, page_size=64, device="cuda"):
    """A zeroed pool of `pages` cache pages of page_size slots and Hk KV heads."""
    if page_size not in PAGE_SIZES:
        raise ValueError(f"page_size must be one of {PAGE_SIZES}, got {page_size}")
    codes = [torch.zeros((pages, Hk, page_size, 128), dtype=torch.uint8, device=device)
             .view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones((pages, Hk), dtype=torch.float32, device=device) for _ in range(2)]
    pos = torch.full((pages, Hk, page_size), -1, dtype=torch.int32, device=device)
    weight = torch.zeros((pages, Hk, page_size), dtype=torch.float32, device=device)
    return KvCache(*codes, *scales, pos, weight)


def kda_cache_append(cache, k, v, block_table, lens, cu_seqlens=None, positions=None,
                     stream=None):
    """Appends the rows k, v [T_total, Hk, 128] bf16 of N sequences (cu_seqlens, or
    equal shares) to their pages, block_table int32 [N, width], after the lens[n]
    slots in use (lens is not changed: add the new rows yourself).  positions:
    int32 [T_total], default the slot numbers.  Returns cache."""
    b = _binding or load_binding()
    _run(stream, "kda_cache_append", b.cache_append, *cache, k, v, block_table, lens, cu_seqlens,
         positions)
    return cache


def kda_cache_attn(cache, q, block_table, lens, scale, cap=0.0, slopes=None, cu_seqlens=None,
                   positions=None, accumulate=False, out=None, workspace=None, stream=None):
    """Attention of the query rows q [T_total, H, 128] bf16 of N sequences
    (cu_seqlens, or equal shares) over the lens[n] cached slots of each, the
    queries' own tokens among them.  A query sees positions up to its own;
    positions int32 [T_total], default: the queries are the newest tokens.
    accumulate: adds the softmax weight of every slot to cache.weight.
    Returns out [T_total, H, 128]."""
    b = _binding or load_binding()
    return _run(stream, "kda_cache_attn", b.cache_attn, *cache, q, block_table, lens, scale, cap,
                slopes, cu_seqlens, positions, accumulate, out, workspace)


def kda_cache_evict(cache, block_table, lens, dst_table, budget, recent, new_lens=None,
                    workspace=None, stream=None):
    """Keeps at most `budget` slots of every sequence and KV head, the newest
    `recent` and those of largest accumulated weight, packed into the pages of
    dst_table int32 [N, dst_width] (other pages than block_table's).  Returns
    new_lens int32 [N] = min(lens, budget); the old pages are free afterwards."""
    b = _binding or load_binding()
    return _run(stream, "kda_cache_evict", b.cache_evict, *cache, block_table, lens, dst_table,
                budget, recent, new_lens, workspace)


def kda_cache_reserve(block_table, lens, new_rows, free_pages, free_count, page_size, rows=None,
                      new_lens=None, cu_seqlens=None, slots=None, new_free_count=None, stream=None):
    """Pages for new_rows int32 [N] more slots of every sequence: taken from the end of
    the free list (free_pages int32 [pages], a place for every page of the pool; the first
    free_count int32 [1] are free) and entered in block_table int32 [N, width], in the order
    of the sequences.  A sequence that the list or its row of the table has no room for
    gets none; its rows must not be appended.  (Without them: the rows with slots >= 0 first,
    packed by the sums of the new lengths less the old.)  rows: the new rows of the call's
    packed tensors, for their slots (None: no slots).  new_lens may be lens, new_free_count free_count; without them the results
    are new tensors.  Returns a Reservation."""
    b = _binding or load_binding()
    return Reservation(*_run(stream, "kda_cache_reserve", b.cache_reserve, block_table, lens, new_rows,
                             free_pages, free_count, page_size, rows, new_lens, cu_seqlens, slots,
                             new_free_count))


def kda_cache_release(block_table, lens, free_pages, free_count, page_size, keep=None,
                      new_free_count=None, stream=None):
    """Gives the pages behind each sequence's first keep int32 [N] slots (None: all of its
    lens[n] slots' pages) back to the free list, in place; the table stays as it is.
    Returns the pages free then, int32 [1] (new_free_count, which may be free_count)."""
    b = _binding or load_binding()
    return _run(stream, "kda_cache_release", b.cache_release, block_table, lens, free_pages, free_count,
                page_size, keep, new_free_count)
