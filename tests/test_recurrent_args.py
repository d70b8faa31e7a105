"""Refusals of the short convolution, the state-space recurrence and the page tables (no GPU
needed): every bad argument returns its status before the device is touched."""
import ctypes

import pytest
import torch

import chunked_gated_delta_11_gb300 as kda
import recurrent_ref as ref
from chunked_gated_delta_11_gb300 import recurrent

FAKE = 1 << 30  # aligned, never dereferenced: validation fails first
FAR = 1 << 34   # apart from what lies at FAKE
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    kda.build.build()
    return kda.load()


def conv(lib, *, opts=True, stride=0, x=FAKE, w=FAKE, bias=None, init=None, cu=None, T=64, C=64, W=4, N=1, out=FAR,
         fin=None):
    o = recurrent._ConvOptions(stride, 1)
    return lib.kda_conv_fwd(ctypes.byref(o) if opts else None, x, w, bias, init, cu, T, C, W, N, out, fin, None)


@pytest.mark.parametrize("kw,status", [
    (dict(opts=False), INVALID),
    (dict(W=1), UNSUPPORTED), (dict(W=5), UNSUPPORTED), (dict(C=12), UNSUPPORTED),
    (dict(C=0), INVALID), (dict(C=-8), INVALID), (dict(N=0), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID),
    (dict(T=65, N=2), INVALID), (dict(cu=FAKE + 2), INVALID),
    (dict(stride=56), INVALID), (dict(stride=68), INVALID), (dict(stride=-64), INVALID),
    (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(out=0), INVALID),
    (dict(x=FAKE + 8), INVALID), (dict(w=FAKE + 8), INVALID), (dict(bias=FAKE + 2), INVALID), (dict(out=FAR + 4), INVALID),
    (dict(init=FAR + 2), INVALID), (dict(fin=FAR + 8), INVALID),
    (dict(out=FAKE + 64 * 128 - 16), INVALID),             # over the last row of x
    (dict(stride=1024, out=FAKE + 1024), INVALID),         # between its rows
    (dict(init=FAKE * 2, fin=FAKE * 2 + 16), INVALID),     # neither in place nor apart
    (dict(fin=FAR + 16), INVALID), (dict(init=FAR + 16), INVALID),   # a state over the output
    (dict(fin=FAKE + 64 * 128 - 16), INVALID),             # over x
])
def test_conv_rejects(lib, kw, status):
    assert conv(lib, **kw) == status


def ssm(lib, *, entry="kda_ssm_step", opts=True, strides=(0, 0, 0, 0), skip=None, bias=None, dtype=0, x=FAKE, dt=FAKE,
        A=FAKE, B=FAKE, C=FAKE, init=None, cu=None, T=64, H=4, G=2, N=1, P=64, S=128, out=FAR, fin=None, ws=()):
    o = recurrent._SsmOptions(*strides, skip, bias, dtype)
    return getattr(lib, entry)(ctypes.byref(o) if opts else None, x, dt, A, B, C, init, cu, T, H, G, N, P, S, out, fin,
                               *ws, None)


BAD_SSM = [
    (dict(opts=False), INVALID),
    (dict(P=32), UNSUPPORTED), (dict(P=96), UNSUPPORTED), (dict(S=16), UNSUPPORTED), (dict(S=256), UNSUPPORTED),
    (dict(H=0), INVALID), (dict(G=0), INVALID), (dict(H=5), INVALID), (dict(H=70000, G=1), INVALID), (dict(N=0), INVALID),
    (dict(N=1 << 22), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(T=65, N=2), INVALID),
    (dict(cu=FAKE + 1), INVALID), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
    (dict(strides=(248, 0, 0, 0)), INVALID), (dict(strides=(260, 0, 0, 0)), INVALID), (dict(strides=(0, 3, 0, 0)), INVALID),
    (dict(strides=(0, 0, 252, 0)), INVALID), (dict(strides=(0, 0, 0, -256)), INVALID),
    (dict(x=0), INVALID), (dict(dt=0), INVALID), (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID),
    (dict(out=0), INVALID), (dict(x=FAKE + 8), INVALID), (dict(dt=FAKE + 1), INVALID), (dict(A=FAKE + 2), INVALID),
    (dict(B=FAKE + 2), INVALID), (dict(C=FAKE + 8), INVALID), (dict(out=FAR + 8), INVALID), (dict(skip=FAKE + 2), INVALID),
    (dict(bias=FAKE + 1), INVALID), (dict(init=FAKE + 4), INVALID), (dict(fin=FAKE + 4), INVALID),
    (dict(init=FAR * 2, fin=FAR * 2 + 64), INVALID), (dict(out=FAKE + 16), INVALID), (dict(fin=FAR + 16), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_SSM)
def test_ssm_step_rejects(lib, kw, status):
    assert ssm(lib, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_SSM + [(dict(T=(1 << 31) - 128, H=2, G=1), INVALID)])
def test_ssm_fwd_rejects(lib, kw, status):
    assert ssm(lib, entry="kda_ssm_fwd", ws=(None, 0), **kw) == status


def test_ssm_workspace(lib):
    size = kda.kda_ssm_workspace_size
    assert size(256 * 4096, 64, 8, 256, 64, 128) == 0   # enough sequences: none is cut
    need = size(8192, 4, 2, 1, 64, 128)
    assert need > 0
    for bad in (need - 1, 0):
        assert ssm(lib, entry="kda_ssm_fwd", T=8192, ws=(FAKE, bad)) == WORKSPACE
    assert ssm(lib, entry="kda_ssm_fwd", T=8192, ws=(FAKE + 8, need)) == WORKSPACE
    assert size(-1, 4, 2, 1, 64, 128) == 0 and size(64, 4, 3, 1, 64, 128) == 0 and size(64, 4, 2, 1, 80, 128) == 0


@pytest.mark.parametrize("entry,ws", [("kda_ssm_step", ()), ("kda_ssm_fwd", (None, 0))])
@pytest.mark.parametrize("kw", [
    dict(x=FAKE * 2, fin=FAKE * 2), dict(dt=FAKE * 2, fin=FAKE * 2), dict(B=FAKE * 2, fin=FAKE * 2),
    dict(C=FAKE * 2, fin=FAKE * 2 - 65536 * 2 + 16),      # its last 16 bytes
    # rows whose offsets would pass 64 bits
    *(dict(T=1 << 30, out=1 << 45, strides=tuple(i == k and 1 << 40 for k in range(4))) for i in range(4)),
])
def test_ssm_rejects_states_over_inputs_and_endless_rows(lib, entry, ws, kw):
    assert ssm(lib, entry=entry, ws=ws, **kw) == INVALID


def test_conv_rejects_endless_rows(lib):
    assert conv(lib, T=1 << 30, stride=1 << 40, out=1 << 45) == INVALID


def reserve(lib, *, table=FAKE, width=8, lens=FAKE + (1 << 20), new=FAKE + (2 << 20), free=FAKE + (3 << 20),
            count=FAKE + (4 << 20), pages=64, page=64, T=128, N=4, new_lens=FAR, cu=FAR + (1 << 20), slots=FAR + (2 << 20),
            left=FAR + (3 << 20)):
    return lib.kda_cache_reserve(table, width, lens, new, free, count, pages, page, T, N, new_lens, cu, slots, left, None)


LENS, NEW, FREE, COUNT = (FAKE + (i << 20) for i in range(1, 5))


@pytest.mark.parametrize("kw,status", [
    (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(N=16385), UNSUPPORTED),
    (dict(N=0), INVALID), (dict(width=0), INVALID), (dict(pages=-1), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID),
    (dict(width=1 << 25), INVALID),
    (dict(table=0), INVALID), (dict(lens=0), INVALID), (dict(new=0), INVALID), (dict(free=0), INVALID), (dict(count=0), INVALID),
    (dict(new_lens=0), INVALID), (dict(cu=0), INVALID), (dict(left=0), INVALID),
    (dict(table=FAKE + 2), INVALID), (dict(lens=FAKE + 2), INVALID), (dict(slots=FAR + 8), INVALID), (dict(cu=FAR + 2), INVALID),
    (dict(new_lens=LENS + 4), INVALID),                    # neither in place nor apart
    (dict(new_lens=NEW), INVALID), (dict(cu=LENS), INVALID), (dict(slots=LENS), INVALID), (dict(left=FREE), INVALID),
    (dict(table=FREE), INVALID), (dict(left=FAR + 4), INVALID), (dict(cu=FAR), INVALID), (dict(table=LENS - 4), INVALID),
])
def test_reserve_rejects(lib, kw, status):
    assert reserve(lib, **kw) == status


def release(lib, *, table=FAKE, width=8, lens=LENS, keep=None, free=FREE, count=COUNT, pages=64, page=64, N=4, left=FAR):
    return lib.kda_cache_release(table, width, lens, keep, free, count, pages, page, N, left, None)


@pytest.mark.parametrize("kw,status", [
    (dict(page=0), UNSUPPORTED), (dict(N=20000), UNSUPPORTED), (dict(N=-1), INVALID), (dict(width=-1), INVALID),
    (dict(pages=-4), INVALID), (dict(table=0), INVALID), (dict(lens=0), INVALID), (dict(free=0), INVALID),
    (dict(count=0), INVALID), (dict(left=0), INVALID), (dict(keep=FAKE + 1), INVALID), (dict(left=FAR + 1), INVALID),
    (dict(free=LENS), INVALID), (dict(free=FAKE + 16), INVALID), (dict(keep=FREE), INVALID), (dict(left=LENS), INVALID),
    (dict(count=FREE + 4), INVALID),
])
def test_release_rejects(lib, kw, status):
    assert release(lib, **kw) == status


def test_the_binding_refuses_what_is_not_on_a_gpu(lib):
    if not kda.build.binding_built_for():
        pytest.skip("the binding is not built")
    x, w = torch.zeros(4, 8).bfloat16(), torch.zeros(8, 4).bfloat16()
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_conv_fwd(x, w)
    with pytest.raises(TypeError, match="bfloat16"):
        kda.kda_conv_fwd(x.float(), w)
    with pytest.raises(ValueError, match="T_total"):
        kda.kda_ssm_fwd(x, x, w, x, x)
    with pytest.raises(TypeError, match="Tensor"):
        kda.kda_cache_release([[0]], w, w, w, 64)


# ------------------------------------------------------------------ the 64-bit forms themselves

def test_the_chunked_form_is_the_recurrence():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    lengths, H, G, P, S = [130, 0, 1, 260], 3, 1, 4, 5
    T = sum(lengths)
    a = (r(T, H, P), r(T, H), -torch.rand(H, generator=g) * 3, r(T, G, S), r(T, G, S), r(H), r(H), r(4, H, P, S), lengths)
    y0, _, m0, _ = ref.ssm_step(*a)
    y1, _, m1, _ = ref.ssm_chunks(*a)
    assert (y0 - y1).abs().max() < 1e-11 and (m0 - m1).abs().max() < 1e-11


def test_a_mistake_shows_in_the_chunked_form():
    """The tolerance is narrow enough to see a weight that is one token off."""
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    T, H, P, S = 200, 2, 8, 16
    x, dt, A, B, C = r(T, H, P), r(T, H), -torch.rand(H, generator=g) * 3, r(T, 1, S), r(T, 1, S)
    y, tol, m, mtol = ref.ssm_chunks(x, dt, A, B, C, None, None, None, [T])
    shifted = torch.cat([dt[1:], dt[-1:]])
    y2, _, m2, _ = ref.ssm_chunks(x, shifted, A, B, C, None, None, None, [T])
    assert ((y - y2).abs() > tol).double().mean() > 0.3 and ((m - m2).abs() > mtol).double().mean() > 0.9
