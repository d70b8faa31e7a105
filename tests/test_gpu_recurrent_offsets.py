"""Rows and states whose element offsets pass 32 bits: the last sequence of a large call against the
same sequence in a call of its own."""
import pytest
import torch

import chunked_gated_delta_11_gb300 as kda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    kda.build.build()
    kda.load()


@pytest.fixture(autouse=True)
def _room():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    yield
    torch.cuda.empty_cache()


def randn(g, *shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def far_rows(g, T, row):
    """T rows of `row` elements, 2^26 apart."""
    wide = torch.empty((T - 1) * (1 << 26) + row, dtype=torch.bfloat16, device="cuda")
    rows = wide.as_strided((T, row), (1 << 26, 1))
    rows.copy_(randn(g, T, row))
    return rows


def test_conv_rows():
    g = torch.Generator(device="cuda").manual_seed(0)
    T, C, N = 70000, 32768, 7
    assert T * C > 1 << 31
    x, w, state = randn(g, T, C), randn(g, C, 4), randn(g, N, 3, C)
    out, fin = kda.kda_conv_fwd(x, w, initial_state=state, N=N)
    last, end = kda.kda_conv_fwd(x[-T // N:], w, initial_state=state[-1:])
    assert torch.equal(out[-T // N:], last) and torch.equal(fin[-1:], end)
    x = far_rows(g, 40, 520)
    out, fin = kda.kda_conv_fwd(x, w[:520], N=2)
    near, end = kda.kda_conv_fwd(x.contiguous(), w[:520], N=2)
    assert torch.equal(out, near) and torch.equal(fin, end)
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("entry", ["kda_ssm_fwd", "kda_ssm_step"])
def test_ssm_rows(entry):
    g = torch.Generator(device="cuda").manual_seed(1)
    call = getattr(kda, entry)
    N, H, P, S = 35, 512, 64, 64
    T = 2000 * N
    assert T * H * P > 1 << 31
    x, dt, B, C = randn(g, T, H, P), randn(g, T, H), randn(g, T, 1, S), randn(g, T, 1, S)
    A = -torch.rand(H, generator=g, device="cuda")
    out, fin = call(x, dt, A, B, C, N=N)
    r = slice(T - 2000, T)
    last, end = call(x[r], dt[r], A, B[r], C[r])
    assert torch.equal(out[r], last) and torch.equal(fin[-1:], end)
    # strided ones
    T, H, n = 48, 4, 4 * P
    rows = far_rows(g, T, n + 2 * S + H)
    a = (rows[:, :n].view(T, H, P), rows[:, n + 2 * S:], A[:H], rows[:, n:n + S].view(T, 1, S), rows[:, n + S:n + 2 * S].view(T, 1, S))
    out, fin = call(*a, N=3)
    near, end = call(*[t.contiguous() for t in a], N=3)
    assert torch.equal(out, near) and torch.equal(fin, end)
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("entry", ["kda_ssm_fwd", "kda_ssm_step"])
def test_ssm_states(entry):
    g = torch.Generator(device="cuda").manual_seed(2)
    call = getattr(kda, entry)
    N, H, P, S = 3000, 96, 64, 128
    assert N * H * P * S > 1 << 31
    x, dt, B, C = randn(g, N, H, P), randn(g, N, H), randn(g, N, 1, S), randn(g, N, 1, S)
    A = -torch.rand(H, generator=g, device="cuda")
    m = torch.empty((N, H, P, S), device="cuda").normal_(generator=g)
    old = m[-2:].clone()
    out, fin = call(x, dt, A, B, C, initial_state=m, N=N, final_state=m)
    last, end = call(x[-2:], dt[-2:], A, B[-2:], C[-2:], initial_state=old, N=2)
    assert torch.equal(out[-2:], last) and torch.equal(fin[-2:], end)
    assert kda.kda_device_status() == 0
