"""Decays of the state-space scan far from 1 on the GPU, against the 64-bit forms of recurrent_ref."""
import pytest
import torch

import chunked_gated_delta_11_gb300 as kda
import recurrent_ref as ref
from test_gpu_recurrent import check_ssm, gen, randn, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    kda.build.build()
    kda.load()


def quiet(lengths, busy, sums, S, state):
    """Rows that add nothing to the states but for those in `busy` of every sequence; head h decays by
    e^{sums[h]} in 128 tokens."""
    g, T, H = gen(sum(lengths)), sum(lengths), len(sums)
    x, B, C = randn(g, T, H, 64), randn(g, T, 1, S), randn(g, T, 1, S)
    at = 0
    for n in lengths:
        x[at:at + n][[t not in busy for t in range(n)]] = 0
        at += n
    dt = torch.full((T, H), -1.0, dtype=torch.bfloat16)
    d = torch.nn.functional.softplus(torch.tensor(-1.0, dtype=torch.float64))
    init = torch.randn((len(lengths), H, 64, S), generator=g) if state else None
    return x, dt, (torch.tensor(sums, dtype=torch.float64) / (128 * d)).float(), B, C, None, None, init


@pytest.mark.parametrize("lengths", [[128], [384, 100, 129]])
@pytest.mark.parametrize("S", [64, 128])
def test_what_is_left_of_a_state_that_only_decays(lengths, S):
    check_ssm("kda_ssm_fwd", quiet(lengths, (), [-0.2, -4.0, -8.0, -12.0, -14.0, -16.0, -20.0], S, True), lengths)
    check_ssm("kda_ssm_fwd", quiet(lengths, range(20), [-0.5, -6.0, -10.0, -16.0], S, True), lengths)


@pytest.mark.parametrize("busy", [range(0, 128), range(1000, 1300)])
def test_what_is_left_of_it_in_pieces(busy):
    sums = [-0.1, -1.0, -2.0, -3.0, -4.0]
    assert kda.kda_ssm_workspace_size(2048, len(sums), 1, 1, 64, 128) > 0
    check_ssm("kda_ssm_fwd", quiet([2048], busy, sums, 128, False), [2048])
    if busy[0]:  # (of what the first rows add, the strongest of these would leave less than a float can hold)
        sums = [-4.0, -6.0, -8.0, -10.0, -12.0]
        check_ssm("kda_ssm_fwd", quiet([2048], busy, sums, 128, False), [2048])


def strong(rates, pattern, T):
    """One sequence of small random rows; head h has A = -rates[h], token t the step size that gives
    softplus(dt) of pattern[t % len(pattern)]."""
    g, H = gen(T + len(pattern)), len(rates)
    dt = torch.tensor(pattern).repeat(T // len(pattern) + 1)[:T, None].expand(T, H).to(torch.bfloat16).contiguous()
    return randn(g, T, H, 64), dt, -torch.tensor(rates), randn(g, T, 1, 64), randn(g, T, 1, 64), None, None, None


def narrow(x, dt, A, B, C, T, CHUNK=ref.CHUNK):
    """(out, tolerance) of one sequence of T <= 128 rows from a zero state, every weight with errors of
    its own: of the step sizes between its two tokens (e_d, and three roundings to the logarithm), of
    14 additions and a difference of sums since the start of the row's 32 where the tokens share
    them (a token's part there is at most 128 ln 2: less than that is left of nothing), of 20
    roundings of the exponent itself elsewhere, of two exponentials and three products; then
    the rounding to bf16, S products and T additions that may cut off, and the output's own."""
    assert T <= CHUNK
    F, BF = ref.F32, ref.BF16
    d, ed = ref._steps(dt, A, None)
    x, B, C, A = (t.double() for t in (x, B[:, 0], C[:, 0], A))
    s = (A * d).T                                                            # [H, T]
    l = torch.cumsum(s, 1)
    D = l[:, :, None] - l[:, None]
    D = torch.where(torch.ones(T, T, dtype=torch.bool).tril(), D, -torch.inf)
    eD = torch.cumsum((s.abs() * (ed.T + 3 * F)), 1)
    eD = (eD[:, :, None] - eD[:, None]).clamp(min=0)
    block = torch.arange(T) // 32
    same = block[:, None] == block[None]
    most = s.abs().clamp(max=128 * 0.6931472)
    upto = torch.stack([most[:, 32 * b:t + 1].sum(1) for t, b in enumerate(block.tolist())], 1)   # [H, T]
    own = torch.eye(T, dtype=torch.bool)
    e = eD + torch.where(same, torch.where(own, 0.0, 16 * F * upto[:, :, None]), 20 * F * D.abs().nan_to_num(posinf=0.0))
    e = torch.expm1(e.clamp(max=20.0)) + 2.0 ** -20 + ed.T[:, None]
    W = torch.exp(D) * d.T[:, None]
    S, Sa = C @ B.T, C.abs() @ B.abs().T
    X = x.transpose(0, 1)
    y = (W * S) @ X
    tol = (W * (S.abs() * (BF + e) + B.shape[1] * 2.0 ** -23 * Sa)) @ X.abs() + T * 2.0 ** -23 * ((W * S).abs() @ X.abs())
    # weights below the least normal float are none
    tol = tol + 2.0 ** -125 * (d.T[:, None] * Sa) @ X.abs()
    return y.transpose(0, 1), (tol + BF * (y.abs() + tol)).transpose(0, 1)


@pytest.mark.parametrize("T", [1, 33, 128])
@pytest.mark.parametrize("pattern", [
    (-1.0,),                                   # every token leaves nothing of the ones before
    (1000.0, -3.0, -2.0, -4.0, -5.0, -3.0, -2.5, -3.5, -4.0),   # one in nine does
    (50.0, -6.0), (-6.0,) * 40 + (300.0,)])
def test_weights_beside_tokens_that_leave_nothing(T, pattern):
    rates = [0.5, 30.0, 1e3, 1e4, 1e5, 1e6]
    x, dt, A, B, C, *_ = case = strong(rates, pattern, T)
    out, _ = kda.kda_ssm_fwd(*[None if t is None else t.cuda() for t in case])
    step, _ = kda.kda_ssm_step(*[None if t is None else t.cuda() for t in case])
    assert kda.kda_device_status() == 0
    want, tol = narrow(x, dt, A, B, C, T)
    plain, plain_tol, _, _ = ref.ssm_step(*case, [T])
    assert (plain - want).abs().max() <= 1e-9 * want.abs().max()
    within(step, plain, plain_tol, "token by token")
    within(out, want, tol, "out")
