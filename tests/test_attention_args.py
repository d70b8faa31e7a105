"""Refusals of the softmax-attention entry points (no GPU needed): every bad
argument returns its status before the device is touched."""
import ctypes

import pytest
import torch

import attn_ref as ref
import chunked_gated_delta_11_gb300 as kda
from chunked_gated_delta_11_gb300 import attention

FAKE = 1 << 20  # aligned, never dereferenced: validation fails first
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    kda.build.build()
    return kda.load()


def attn(lib, *, opts=True, mask=1, cap=0.0, slopes=None, prefix=None, q=FAKE, k=FAKE, v=FAKE, scale=0.1, cu=None,
         T=64, H=4, Hk=2, N=1, D=128, out=FAKE):
    o = attention._AttnOptions(mask, cap, slopes, prefix)
    return lib.kda_attn_fwd(ctypes.byref(o) if opts else None, q, k, v, scale, cu, T, H, Hk, N, D, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(opts=False), INVALID),
    (dict(mask=3), INVALID), (dict(mask=-1), INVALID),
    (dict(mask=2), INVALID),                       # a prefix mask without prefix_lens
    (dict(mask=1, prefix=FAKE), INVALID),          # prefix_lens without a prefix mask
    (dict(mask=2, prefix=FAKE + 2), INVALID),
    (dict(cap=-1.0), INVALID), (dict(cap=float("inf")), INVALID), (dict(cap=float("nan")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(slopes=FAKE + 2), INVALID),
    (dict(D=64), UNSUPPORTED),
    (dict(H=0), INVALID), (dict(Hk=0), INVALID), (dict(H=5, Hk=2), INVALID), (dict(H=70000, Hk=70000), INVALID),
    (dict(N=0), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(T=65, N=2), INVALID),
    (dict(cu=FAKE + 2), INVALID),
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(out=0), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(k=FAKE + 2), INVALID), (dict(v=FAKE + 4), INVALID), (dict(out=FAKE + 8), INVALID),
    (dict(T=0, q=0, k=0, v=0, out=0), 0),          # nothing to do
])
def test_attn_fwd(lib, kw, status):
    assert attn(lib, **kw) == status


def pool(**kw):
    f = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, pos=FAKE, weight=FAKE, pages=8, page_size=64, Hk=2, D=128)
    f.update(kw)
    return attention._Cache(*(f[n] for n, _ in attention._Cache._fields_))


BAD_POOLS = [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(k_scale=0), INVALID), (dict(v_scale=0), INVALID),
    (dict(pos=0), INVALID), (dict(weight=0), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 1), INVALID),
    (dict(k_scale=FAKE + 2), INVALID), (dict(pos=FAKE + 4), INVALID), (dict(weight=FAKE + 4), INVALID),
    (dict(pages=0), INVALID), (dict(pages=-1), INVALID), (dict(Hk=0), INVALID), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=256), UNSUPPORTED), (dict(page_size=0), UNSUPPORTED), (dict(D=64), UNSUPPORTED),
    (dict(pages=(1 << 31) - 1, Hk=60000), INVALID),
]


def append(lib, cache=None, k=FAKE, v=FAKE, table=FAKE, width=4, lens=FAKE, positions=None, cu=None, T=8, N=2):
    c = cache if cache is not None else pool()
    return lib.kda_cache_append(ctypes.byref(c), k, v, table, width, lens, positions, cu, T, N, None)


def cached(lib, cache=None, cap=0.0, slopes=None, positions=None, accumulate=0, q=FAKE, scale=0.1, table=FAKE, width=4,
           lens=FAKE, cu=None, T=8, H=4, N=2, out=FAKE, ws=None, ws_bytes=0, opts=True):
    c = cache if cache is not None else pool()
    o = attention._CacheAttnOptions(cap, slopes, positions, accumulate)
    return lib.kda_cache_attn(ctypes.byref(o) if opts else None, ctypes.byref(c), q, scale, table, width, lens, cu, T, H,
                              N, out, ws, ws_bytes, None)


def evict(lib, cache=None, table=FAKE, width=4, lens=FAKE, dst=FAKE, dst_width=2, budget=100, recent=10, N=2,
          new_lens=FAKE, ws=None, ws_bytes=0):
    c = cache if cache is not None else pool()
    return lib.kda_cache_evict(ctypes.byref(c), table, width, lens, dst, dst_width, budget, recent, N, new_lens, ws,
                               ws_bytes, None)


@pytest.mark.parametrize("call", [append, cached, evict])
@pytest.mark.parametrize("kw,status", BAD_POOLS)
def test_pools(lib, call, kw, status):
    assert call(lib, cache=pool(**kw)) == status


@pytest.mark.parametrize("call", [append, cached, evict])
@pytest.mark.parametrize("kw", [dict(table=0), dict(lens=0), dict(table=FAKE + 2), dict(lens=FAKE + 1), dict(width=0),
                                dict(width=-3), dict(N=0), dict(width=(1 << 31) - 1), dict(N=(1 << 31) - 2)])
def test_tables(lib, call, kw):
    assert call(lib, **kw) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(positions=FAKE + 2), INVALID), (dict(cu=FAKE + 2), INVALID), (dict(T=9), INVALID), (dict(T=-2), INVALID),
    (dict(T=0, k=0, v=0), 0),
])
def test_append(lib, kw, status):
    assert append(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(opts=False), INVALID), (dict(cap=-2.0), INVALID), (dict(cap=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(slopes=FAKE + 1), INVALID), (dict(positions=FAKE + 2), INVALID),
    (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 2), INVALID),
    (dict(H=3), INVALID), (dict(H=0), INVALID), (dict(T=9), INVALID), (dict(cu=FAKE + 2), INVALID),
    (dict(T=1 << 30, H=4), INVALID),
    (dict(ws=FAKE, ws_bytes=16, accumulate=1), WORKSPACE), (dict(ws=FAKE + 8, ws_bytes=1 << 40, accumulate=1), WORKSPACE),
    (dict(T=0, q=0, out=0), 0),
])
def test_cache_attn(lib, kw, status):
    assert cached(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dst=0), INVALID), (dict(dst=FAKE + 2), INVALID), (dict(dst_width=0), INVALID), (dict(new_lens=0), INVALID),
    (dict(budget=0), INVALID), (dict(budget=-5), INVALID), (dict(recent=-1), INVALID), (dict(recent=101), INVALID),
    (dict(ws=FAKE, ws_bytes=16), WORKSPACE), (dict(ws=FAKE + 4, ws_bytes=1 << 40), WORKSPACE),
])
def test_evict(lib, kw, status):
    assert evict(lib, **kw) == status


def test_workspace_sizes(lib):
    c = pool()
    assert lib.kda_cache_evict_workspace_size(ctypes.byref(c), 2, 100) == 1792   # 2 x 2 x 100 int32, rounded to 256
    assert lib.kda_cache_evict_workspace_size(ctypes.byref(c), 0, 100) == 0
    assert lib.kda_cache_evict_workspace_size(ctypes.byref(pool(D=64)), 2, 100) == 0
    size = lambda T, H, acc: lib.kda_cache_attn_workspace_size(ctypes.byref(c), T, H, 2, 4, acc)  # noqa: E731
    assert size(2, 4, 1) >= 2 * 4 * 4
    assert size(2, 5, 0) == 0 and size(0, 4, 1) == 0


def test_binding_checks_its_tensors(lib):
    q = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_attn_fwd(q, q, q, 0.1)
    with pytest.raises(TypeError, match="bfloat16"):
        kda.kda_attn_fwd(q.float(), q, q, 0.1)
    with pytest.raises(TypeError, match="Tensor"):
        kda.kda_attn_fwd(None, q, q, 0.1)
    with pytest.raises(ValueError, match="mask"):
        kda.kda_attn_fwd(q, q, q, 0.1, mask="window")
    with pytest.raises(ValueError, match="T_total"):
        kda.kda_attn_fwd(q[0], q, q, 0.1)
    with pytest.raises(ValueError, match="page_size"):
        kda.kda_cache_alloc(4, 2, 48, device="cpu")
    cache = kda.kda_cache_alloc(4, 2, 16, device="cpu")
    assert cache.k.dtype == torch.float8_e4m3fn and cache.k.shape == (4, 2, 16, 128)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: kda.kda_cache_append(cache, q, q, table, lens),
                 lambda: kda.kda_cache_attn(cache, q, table, lens, 0.1),
                 lambda: kda.kda_cache_evict(cache, table, lens, table, 4, 1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_the_references_own_rounding():
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(50_000, generator=g) * torch.exp(4 * torch.randn(50_000, generator=g))).clamp(-448, 448)
    assert torch.equal(ref.to_codes(x.double()), x.to(torch.float8_e4m3fn).double())
    assert [ref.exponent(a) for a in (0.0, 448.0, 448.1, 3.5, 3.51, 1e38)] == [-64, 0, 1, -7, -6, 118]
