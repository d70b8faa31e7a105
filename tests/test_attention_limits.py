"""Refusals of the softmax-attention entry points at the limits of their contracts (no GPU needed)."""
import ctypes

import pytest

import chunked_gated_delta_11_gb300 as kda
from chunked_gated_delta_11_gb300 import attention

FAKE = 1 << 20  # aligned, never dereferenced: validation fails first
INVALID, WORKSPACE = 1, 3


@pytest.fixture(scope="module")
def lib():
    kda.build.build()
    return kda.load()


def pool():
    return attention._Cache(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8, 64, 2, 128)


def evict(lib, lens=FAKE, new_lens=FAKE, budget=100, recent=10, N=4, ws=None, ws_bytes=0):
    return lib.kda_cache_evict(ctypes.byref(pool()), FAKE, 4, lens, FAKE, 2, budget, recent, N, new_lens, ws, ws_bytes,
                               None)


@pytest.mark.parametrize("shift", [4, 12, -4, -12])
def test_evict_refuses_new_lengths_that_overlap_the_old_ones(lib, shift):
    assert evict(lib, new_lens=FAKE + shift) == INVALID


@pytest.mark.parametrize("shift", [0, 16, -16])
def test_evict_takes_lengths_in_place_or_apart(lib, shift):
    # the next check fails, of a workspace that is too small: nothing was launched
    assert evict(lib, new_lens=FAKE + shift, ws=FAKE, ws_bytes=16) == WORKSPACE


def test_evict_needs_no_workspace_beyond_the_tables_slots(lib):
    need = lib.kda_cache_evict_workspace_size(ctypes.byref(pool()), 4, 4 * 64)
    call = lambda size, ws: evict(lib, budget=2 ** 31 - 1, recent=2 ** 31 - 1, ws=ws, ws_bytes=size)  # noqa: E731
    assert call(need - 1, FAKE) == WORKSPACE
    # enough bytes, but too small for another reason: the budget itself is refused
    assert evict(lib, budget=2 ** 31 - 1, recent=-1, ws=FAKE, ws_bytes=need) == INVALID


@pytest.fixture
def own_binding(lib, tmp_path, monkeypatch):
    """The binding's files in a folder of the test's, and nothing loaded."""
    monkeypatch.setattr(kda.build, "BINDING", str(tmp_path / "attn_binding.so"))
    monkeypatch.setattr(kda.build, "BINDING_TAG", str(tmp_path / "attn_binding.tag"), raising=False)
    monkeypatch.setattr(attention, "_binding", None)
    (tmp_path / "libkda.so").symlink_to(kda.build.LIB)
    return tmp_path


def test_the_rest_is_built_where_the_binding_cannot_be(own_binding, monkeypatch):
    def no_headers():
        raise RuntimeError("Python.h: no such file")

    monkeypatch.setattr(kda.build, "_compile_binding", no_headers)
    with pytest.warns(UserWarning, match="Python.h"):
        assert kda.build.build() == kda.build.LIB
    kda.load()
    with pytest.raises(RuntimeError, match="not built"):
        attention.load_binding()


def test_a_binding_of_another_torch_is_not_loaded(own_binding, monkeypatch):
    (own_binding / "attn_binding.so").write_bytes(b"")
    (own_binding / "attn_binding.tag").write_text("torch 2.0.0, cpython-38")
    assert not kda.build.up_to_date()
    with pytest.raises(RuntimeError, match="built for torch 2.0.0"):
        attention.load_binding()
    kda.build.build()
    assert kda.build.up_to_date()
    assert hasattr(attention.load_binding(), "attn_fwd")
