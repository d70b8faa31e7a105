"""What the state-space scan keeps of its states on the GPU: the same for every call that wants
the outputs, all bits of what a token adds, no error that grows with the length."""
import pytest
import torch

import chunked_gated_delta_11_gb300 as kda
import recurrent_ref as ref
from test_gpu_recurrent import cu_of, dev, gen, randn, run_ssm, ssm_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    kda.build.build()
    kda.load()


@pytest.mark.parametrize("lengths,H,G,P,S", [([300, 7, 0, 128], 3, 1, 64, 128), ([500], 2, 2, 128, 64), ([2300], 2, 1, 64, 128)])
def test_outputs_do_not_depend_on_who_wants_the_states(lengths, H, G, P, S):
    case = ssm_case(70, lengths, H, G, P, S, state=None, rate=0.5)
    out, fin = run_ssm("kda_ssm_fwd", case, lengths)
    alone, none = run_ssm("kda_ssm_fwd", case, lengths, output_final_state=False)
    half, fin16 = run_ssm("kda_ssm_fwd", case, lengths,
                          final_state=torch.empty((len(lengths), H, P, S), dtype=torch.bfloat16, device="cuda"))
    assert none is None
    assert torch.equal(out, alone) and torch.equal(out, half)
    assert torch.equal(fin.to(torch.bfloat16), fin16)


def _bits(g, *shape):
    """Floats of every exponent, zeros, infinities, and values halfway between two bf16."""
    v = torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, dtype=torch.int64).to(torch.int32)
    v[..., ::7] = v[..., ::7] & ~0xffff | 0x8000
    v[..., ::11] = v[..., ::11] & ~0xffff
    f = v.view(torch.float32)
    f = torch.where(torch.isnan(f), torch.inf, f)
    f[..., 3], f[..., 4] = 0.0, -0.0
    return f


@pytest.mark.parametrize("P,S", [(64, 128), (128, 128), (64, 64)])
def test_a_state_that_nothing_happens_to_keeps_every_bit(P, S):
    """Step sizes of zero: the state of each chunk is the one before it."""
    lengths, H, G = [384, 0, 1, 200], 2, 1
    g, T = gen(71), sum(lengths)
    x, B, C = randn(g, T, H, P), randn(g, T, G, S), torch.zeros((T, G, S), dtype=torch.bfloat16)
    init = _bits(g, 4, H, P, S)
    case = x, torch.full((T, H), -200.0, dtype=torch.bfloat16), torch.full((H,), -3.0), B, C, None, None, init
    _, fin = run_ssm("kda_ssm_fwd", case, lengths)
    assert torch.equal(fin.cpu(), init)
    # and a NaN in it stays one, in its own channel's outputs too
    init[0, 1, 5, 9], init[3, 0, 2, 1] = float("nan"), torch.tensor(-1, dtype=torch.int32).view(torch.float32)
    init = init.clamp(-1e30, 1e30)
    out, fin = run_ssm("kda_ssm_fwd", (*case[:4], torch.ones_like(C), None, None, init), lengths)
    assert torch.equal(torch.isnan(fin.cpu()), torch.isnan(init))
    bad = torch.isnan(out).cpu()
    assert bad[:384, 1, 5].all() and bad[385:, 0, 2].all() and bad.sum() == 384 + 200


def _tokens(lengths, H, P, S, seed):
    """One token a sequence from a zero state, in rows x whose product with d needs all 24 bits."""
    g, T = gen(seed), sum(lengths)
    x = (1.9921875 * (1 - 2 * torch.randint(0, 2, (T, H, P), generator=g))).to(torch.bfloat16)
    return x, randn(g, T, H), -torch.rand(H, generator=g), randn(g, T, 1, S), randn(g, T, 1, S), None, None, None


def _addends(x, terms):
    """The sum of that many bf16 numbers, each of what the ones before leave."""
    total, left = torch.zeros_like(x), x.clone()
    for _ in range(terms):
        p = left.to(torch.bfloat16).double()
        total, left = total + p, left - p
    return total


@pytest.mark.parametrize("P,S", [(64, 128), (128, 64)])
def test_a_token_adds_all_bits_to_the_state(P, S):
    """d x B^T of one token: d is off by e_d (recurrent_ref), its exponential weight 2^0 by 2^-22, d x
    by a rounding, the three products' sum by a cut of 2^-23 each."""
    N, H = 40, 4
    x, dt, A, B, *_ = case = _tokens([1] * N, H, P, S, 72)
    _, fin = run_ssm("kda_ssm_fwd", case, [1] * N)
    d, ed = ref._steps(dt, A, None)
    dx = d[..., None] * x.double()
    want = dx[..., None] * B.double()[:, :, None]
    rel = (ed + 2.0 ** -22 + ref.F32 + 3 * 2.0 ** -23)[..., None, None]
    assert ((fin.double().cpu() - want).abs() <= rel * want.abs()).all()
    # two addends would not do
    short = _addends(dx.float().double(), 2)[..., None] * B.double()[:, :, None]
    assert ((short - want).abs() > rel * want.abs()).double().mean() > 0.2


@pytest.mark.parametrize("T,H,P,S,A,whole", [
    (8192, 304, 64, 64, 0.0, True), (4096, 152, 128, 128, -1e-5, True), (16384, 2, 64, 128, 0.0, False),
    (16384, 1, 128, 64, -1e-5, False)])
def test_the_error_of_a_state_does_not_grow_with_its_length(T, H, P, S, A, whole):
    """Heads that hardly decay, and states that only grow.  A chunk's sum is cut off 24 times (2^-23 of
    it at most, half of that on average and of half the sum), what it is added to is rounded: by
    2^-24 of the state a chunk, either way, beside the errors of the weights and of the decay."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, B, C = (r(T, H, P).abs().bfloat16(), r(T, 1, S).abs().bfloat16(), r(T, 1, S).bfloat16())
    dt = (0.5 * r(T, H) - 1.0).bfloat16()
    rate = torch.full((H,), A, device="cuda")
    init = r(1, H, P, S).abs()
    assert (kda.kda_ssm_workspace_size(T, H, 1, 1, P, S) == 0) == whole
    _, fin = kda.kda_ssm_fwd(x, dt, rate, B, C, initial_state=init)
    assert kda.kda_device_status() == 0
    d = torch.nn.functional.softplus(dt.double())
    l = torch.cumsum(d * rate.double(), 0)
    w = torch.exp(l[-1:] - l) * d                                    # [T, H]
    add = torch.einsum("thp,ts->hps", w[..., None] * x.double(), B[:, 0].double())
    old = torch.exp(l[-1])[:, None, None] * init[0].double()
    want = old + add
    err = fin[0].double() - want
    chunks = -(-T // ref.CHUNK)
    ed = (8 + dt.double().abs().max().item()) * ref.F32
    # the decay: e_d and a few roundings of all of l, half a step of a factor near 1 and a product a chunk
    decay = -l[-1].min().item() * (ed + 20 * ref.F32) + 2 * chunks * ref.F32
    tol = add * (ed + 2.0 ** -21 + 24 * 2.0 ** -23 + decay) + old * decay + chunks * ref.F32 * want
    assert (err.abs() <= tol).all()
    # no bias: the cuts of a chunk's own sum (24 halves of a step of half of it), the weights' functions
    bias = (err.sum() / want.sum()).item()
    assert abs(bias) <= 12 * 2.0 ** -24 + 8 * 2.0 ** -24
    assert err.norm() <= (ed + 12 * 2.0 ** -24) * want.norm()


@pytest.mark.parametrize("lengths,H,G,P,S", [([2048] * 8, 64, 8, 64, 128), ([1500, 700, 2000, 128] * 3, 32, 1, 128, 64),
                                             ([8192], 64, 8, 64, 128)])
def test_the_same_bits_every_time(lengths, H, G, P, S):
    """Every SM at work for many chunks, other work between the calls."""
    case = [dev(t) for t in ssm_case(73, lengths, H, G, P, S, rate=0.2)]
    cu = cu_of(lengths).cuda()
    call = lambda: kda.kda_ssm_fwd(*case[:-1], initial_state=case[-1], cu_seqlens=cu)  # noqa: E731
    out, fin = call()
    want, state = kda.kda_ssm_step(*case[:-1], initial_state=case[-1], cu_seqlens=cu)
    for got, ref_, tol in ((out, want, 1e-2), (fin, state, 1e-5)):
        assert (got.double() - ref_.double()).norm() <= tol * ref_.double().norm()
    for k in range(12):
        if k % 3 == 2:
            torch.empty(40 << 20, device="cuda").normal_()
        again, fin2 = call()
        assert torch.equal(again, out) and torch.equal(fin2, fin)
    assert kda.kda_device_status() == 0


@pytest.mark.parametrize("entry", ["kda_ssm_fwd", "kda_ssm_step"])
@pytest.mark.parametrize("state", ["fp32", "bf16", None])
def test_a_call_without_rows(entry, state):
    case = ssm_case(74, [0, 0, 0], 3, 1, 64, 128, state)
    out, fin = run_ssm(entry, case, [0, 0, 0])
    assert out.shape == (0, 3, 64)
    assert torch.equal(fin.cpu(), case[-1] if state else torch.zeros(3, 3, 64, 128))
    out, fin = run_ssm(entry, case, [0, 0, 0], output_final_state=False)
    assert out.numel() == 0 and fin is None


@pytest.mark.parametrize("entry", ["kda_ssm_fwd", "kda_ssm_step"])
@pytest.mark.parametrize("at", [200, 255, 256, 300])
def test_what_a_token_that_is_not_finite_reaches(entry, at):
    """Nothing before it but, in the chunks' form and through x alone, its own channel in its chunk."""
    lengths, H, P = [450], 3, 64
    case = ssm_case(75, lengths, H, 1, P, 128, rate=0.5)
    out, _ = run_ssm(entry, case, lengths)
    for which in (1, 3, 4):                       # dt, B, C
        spoilt = [t if t is None else t.clone() for t in case]
        spoilt[which][at] = float("nan")
        got, fin = run_ssm(entry, spoilt, lengths)
        assert torch.equal(got[:at], out[:at])
        assert torch.isnan(got[at]).all()
        assert torch.isnan(fin).all() == (which != 4) and (which != 4 or torch.equal(got[at + 1:], out[at + 1:]))
    spoilt = [t if t is None else t.clone() for t in case]
    spoilt[0][at, 1, 7] = float("inf")
    got, fin = run_ssm(entry, spoilt, lengths)
    chunk = at // ref.CHUNK * ref.CHUNK
    first = chunk if entry == "kda_ssm_fwd" else at
    mine = torch.zeros_like(out, dtype=torch.bool)
    mine[first:, 1, 7] = True
    assert torch.equal(got[~mine], out[~mine])
    assert not torch.isfinite(got[at:, 1, 7]).any() and not torch.isfinite(fin[0, 1, 7]).any()


def test_a_convolution_for_each_of_q_k_and_v():
    """Columns of the projected rows, where they lie: the tensors that the KDA pass takes, without a copy."""
    lengths, H, D = [70, 1, 200], 2, 128
    T, n = sum(lengths), 2 * 128
    g = gen(76)
    rows, taps, held = randn(g, T, 3 * n).cuda(), randn(g, 3 * n, 4).cuda(), randn(g, 3, 3, 3 * n).cuda()
    cu = cu_of(lengths).cuda()
    out, fin = kda.kda_conv_fwd(rows, taps, initial_state=held, cu_seqlens=cu)
    parts = [kda.kda_conv_fwd(rows[:, c], taps[c], initial_state=held[..., c].contiguous(), cu_seqlens=cu)
             for c in (slice(i * n, i * n + n) for i in range(3))]
    for i, (o, f) in enumerate(parts):
        assert o.is_contiguous() and torch.equal(o, out[:, i * n:i * n + n]) and torch.equal(f, fin[..., i * n:i * n + n])
    q, k, v = (o.view(T, H, D) for o, _ in parts)
    gate, beta = randn(g, T, H, D).cuda(), randn(g, T, H).cuda()
    got, state = kda.kda_fwd_fused(q, k, v, gate, beta, D ** -0.5, -5.0, cu_seqlens=cu)
    want, ref_ = kda.kda_fwd_fused(*(t.contiguous() for t in out.view(T, 3, H, D).unbind(1)), gate, beta, D ** -0.5, -5.0,
                                   cu_seqlens=cu)
    assert torch.equal(got, want) and torch.equal(state, ref_) and kda.kda_device_status() == 0
