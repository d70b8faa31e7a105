"""Softmax attention beside the KDA layers: the binding of kda_attn_fwd,
kda_cache_append, kda_cache_attn and kda_cache_evict (include/kda.h).

A hybrid model puts an attention layer after every few KDA layers.  It works on
the same packed rows ([T_total, H, 128] bf16, cu_seqlens), keeps its keys and
values in a paged cache of e4m3 codes with one scale per (page, KV head), and
can drop the cached tokens that got the least attention.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

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


def _api():
    from . import KdaError, load
    return load(), KdaError


def _tensor(t, name, dtype, shape, index):
    """Checks one argument (None in `shape` stands for any size; index: the CUDA
    device) and returns its address.  These checks are a good part of a small call's
    time, so the usual case is one line."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == index and t.is_contiguous() and index >= 0):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    got = t.shape
    if len(got) != len(shape) or any(s is not None and s != g for s, g in zip(shape, got)):
        raise ValueError(f"{name} has shape {tuple(got)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _sizes(t, name, dims, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must be {what}, got {tuple(t.shape)}")
    return t.shape


def _rows(t, name):
    return _sizes(t, name, 3, "[T_total, heads, 128]")


def _table(t, name):
    return _sizes(t, name, 2, "[N, width]")


def _cache(cache, index):
    pages, Hk, page, D = shape = _sizes(cache.k, "cache.k", 4, "[pages, Hk, page_size, 128]")
    f8, f32 = torch.float8_e4m3fn, torch.float32
    blocks, slots = (pages, Hk), (pages, Hk, page)
    return _Cache(_tensor(cache.k, "cache.k", f8, shape, index),
                  _tensor(cache.v, "cache.v", f8, shape, index),
                  _tensor(cache.k_scale, "cache.k_scale", f32, blocks, index),
                  _tensor(cache.v_scale, "cache.v_scale", f32, blocks, index),
                  _tensor(cache.pos, "cache.pos", torch.int32, slots, index),
                  _tensor(cache.weight, "cache.weight", f32, slots, index),
                  pages, page, Hk, D)


def _on(stream, index):
    # the address of torch's current stream, without building a Stream object for it
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """Memory that belongs to the stream it is used on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(workspace, need, like, stream):
    """(tensor to keep, its address, its bytes)"""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _empty(need, torch.uint8, like.device, stream)
        return workspace, workspace.data_ptr(), need
    return workspace, _tensor(workspace, "workspace", torch.uint8, (workspace.numel(),), like.get_device()), workspace.numel()


def _sequences(cu_seqlens, N, index):
    if cu_seqlens is None:
        return None, 1 if N is None else int(N)
    count = _sizes(cu_seqlens, "cu_seqlens", 1, "[N + 1]")[0]
    if N is not None and N != count - 1:
        raise ValueError(f"N is {N}, cu_seqlens has {count - 1} sequences")
    return _tensor(cu_seqlens, "cu_seqlens", torch.int32, (count,), index), count - 1


def kda_attn_fwd(q, k, v, scale, mask="causal", cap=0.0, slopes=None, prefix_lens=None,
                 cu_seqlens=None, N=None, out=None, stream=None):
    """Attention over packed rows: q [T_total, H, 128], k and v [T_total, Hk, 128]
    bf16.  mask: "causal", "full", or "prefix" (the first prefix_lens[n] rows of
    sequence n are seen by all of it); cap: scores become cap * tanh(x / cap);
    slopes: fp32 [H], subtracts slopes[h] * distance.  Returns out [T_total, H, 128]."""
    lib, error = _api()
    T, H, D = _rows(q, "q")
    Hk = _rows(k, "k")[1]
    if mask not in MASKS:
        raise ValueError(f"mask must be one of {tuple(MASKS)}, got {mask!r}")
    dev, bf = q.get_device(), torch.bfloat16
    rows, kv = (T, H, D), (T, Hk, D)
    qp = _tensor(q, "q", bf, rows, dev)
    kp = _tensor(k, "k", bf, kv, dev)
    vp = _tensor(v, "v", bf, kv, dev)
    cu, N = _sequences(cu_seqlens, N, dev)
    if out is None:
        out = _empty(rows, bf, q.device, stream)
    op = _tensor(out, "out", bf, rows, dev)
    opts = _AttnOptions(
        MASKS[mask], cap,
        None if slopes is None else _tensor(slopes, "slopes", torch.float32, (H,), dev),
        None if prefix_lens is None else _tensor(prefix_lens, "prefix_lens", torch.int32, (N,), dev))
    st = lib.kda_attn_fwd(ctypes.byref(opts), qp, kp, vp, scale, cu, T, H, Hk, N, D, op,
                          _on(stream, dev))
    if st:
        raise error(st, "kda_attn_fwd")
    return out


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
    lib, error = _api()
    T, Hk, D = rows = _rows(k, "k")
    N, width = _table(block_table, "block_table")
    dev, bf, i32 = k.get_device(), torch.bfloat16, torch.int32
    c = _cache(cache, dev)
    if Hk != c.Hk:
        raise ValueError(f"k has {Hk} heads, the cache {c.Hk}")
    kp, vp = _tensor(k, "k", bf, rows, dev), _tensor(v, "v", bf, rows, dev)
    table = _tensor(block_table, "block_table", i32, (N, width), dev)
    lp = _tensor(lens, "lens", i32, (N,), dev)
    pp = None if positions is None else _tensor(positions, "positions", i32, (T,), dev)
    cu, N = _sequences(cu_seqlens, N, dev)
    if D != c.D:
        raise ValueError(f"k has {D} channels, the cache {c.D}")
    st = lib.kda_cache_append(ctypes.byref(c), kp, vp, table, width, lp, pp, cu, T, N,
                              _on(stream, dev))
    if st:
        raise error(st, "kda_cache_append")
    return cache


def kda_cache_attn(cache, q, block_table, lens, scale, cap=0.0, slopes=None, cu_seqlens=None,
                   positions=None, accumulate=False, out=None, workspace=None, stream=None):
    """Attention of the query rows q [T_total, H, 128] bf16 of N sequences
    (cu_seqlens, or equal shares) over the lens[n] cached slots of each, the
    queries' own tokens among them.  A query sees positions up to its own;
    positions int32 [T_total], default: the queries are the newest tokens.
    accumulate: adds the softmax weight of every slot to cache.weight.
    Returns out [T_total, H, 128]."""
    lib, error = _api()
    T, H, D = rows = _rows(q, "q")
    N, width = _table(block_table, "block_table")
    dev, bf, i32 = q.get_device(), torch.bfloat16, torch.int32
    c = _cache(cache, dev)
    if D != c.D:
        raise ValueError(f"q has {D} channels, the cache {c.D}")
    qp = _tensor(q, "q", bf, rows, dev)
    table = _tensor(block_table, "block_table", i32, (N, width), dev)
    lp = _tensor(lens, "lens", i32, (N,), dev)
    cu, N = _sequences(cu_seqlens, N, dev)
    if out is None:
        out = _empty(rows, bf, q.device, stream)
    op = _tensor(out, "out", bf, rows, dev)
    opts = _CacheAttnOptions(
        cap, None if slopes is None else _tensor(slopes, "slopes", torch.float32, (H,), dev),
        None if positions is None else _tensor(positions, "positions", i32, (T,), dev),
        1 if accumulate else 0)
    ref = ctypes.byref(c)
    need = lib.kda_cache_attn_workspace_size(ref, T, H, N, width, opts.accumulate)
    keep, ws, nbytes = _workspace(workspace, need, q, stream)
    st = lib.kda_cache_attn(ctypes.byref(opts), ref, qp, scale, table, width, lp, cu, T, H, N, op,
                            ws, nbytes, _on(stream, dev))
    if st:
        raise error(st, "kda_cache_attn")
    return out


def kda_cache_evict(cache, block_table, lens, dst_table, budget, recent, new_lens=None,
                    workspace=None, stream=None):
    """Keeps at most `budget` slots of every sequence and KV head, the newest
    `recent` and those of largest accumulated weight, packed into the pages of
    dst_table int32 [N, dst_width] (other pages than block_table's).  Returns
    new_lens int32 [N] = min(lens, budget); the old pages are free afterwards."""
    lib, error = _api()
    N, width = _table(block_table, "block_table")
    dst_width = _table(dst_table, "dst_table")[1]
    dev, i32 = block_table.get_device(), torch.int32
    c = _cache(cache, dev)
    table = _tensor(block_table, "block_table", i32, (N, width), dev)
    dst = _tensor(dst_table, "dst_table", i32, (N, dst_width), dev)
    lp = _tensor(lens, "lens", i32, (N,), dev)
    if new_lens is None:
        new_lens = _empty((N,), i32, block_table.device, stream)
    np_ = _tensor(new_lens, "new_lens", i32, (N,), dev)
    ref = ctypes.byref(c)
    need = lib.kda_cache_evict_workspace_size(ref, N, budget)
    keep, ws, nbytes = _workspace(workspace, need, block_table, stream)
    st = lib.kda_cache_evict(ref, table, width, lp, dst, dst_width, budget, recent, N, np_, ws,
                             nbytes, _on(stream, dev))
    if st:
        raise error(st, "kda_cache_evict")
    return new_lens
