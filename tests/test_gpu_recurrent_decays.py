"""Decays of the state-space scan far from 1 on the GPU, against the 64-bit forms of recurrent_ref."""
import pytest
import torch

import chunked_gated_delta_11_gb300 as kda
import recurrent_ref as ref
from test_gpu_recurrent import check_ssm, gen, randn

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
