"""The short convolution and the state-space recurrence (both schedules) on the GPU against the
64-bit forms of recurrent_ref."""
import itertools

import pytest
import torch

import chunked_gated_delta_11_gb300 as kda
import recurrent_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    kda.build.build()
    kda.load()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def cu_of(lengths):
    return torch.tensor([0] + list(itertools.accumulate(lengths)), dtype=torch.int32)


def ok():
    assert kda.kda_device_status() == 0


def within(got, want, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    over = ((got - want).abs() - tol).max().item() if got.numel() else 0.0
    assert over <= 0, f"{what}: {over:.3e} over the tolerance"


dev = lambda t: None if t is None else t.cuda()  # noqa: E731


# ------------------------------------------------------------------ convolution

def conv_case(seed, lengths, C, W, bias, state, amp=1.0):
    g = gen(seed)
    x = amp * randn(g, sum(lengths), C)
    return x, randn(g, C, W), randn(g, C) if bias else None, randn(g, len(lengths), W - 1, C) if state else None


def check_conv(case, lengths, silu=True, cu=True, **kw):
    x, w, b, init = case
    out, fin = kda.kda_conv_fwd(dev(x), dev(w), dev(b), initial_state=dev(init),
                                cu_seqlens=cu_of(lengths).cuda() if cu else None, N=None if cu else len(lengths), silu=silu,
                                **kw)
    ok()
    want, tol, state = ref.conv(x, w, b, init, lengths, silu)
    within(out, want, tol, "out")
    assert torch.equal(fin.double().cpu(), state)
    return out, fin


@pytest.mark.parametrize("lengths", [[1], [2, 0, 1], [3, 4, 0, 5], [64], [31, 33, 1, 0, 0, 200], [7, 8, 9, 1, 1, 1, 30], [0, 0]])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("bias,state,silu", [(False, False, True), (True, True, True), (True, True, False)])
def test_conv(lengths, W, bias, state, silu):
    check_conv(conv_case(W + sum(lengths), lengths, 24, W, bias, state), lengths, silu)


@pytest.mark.parametrize("C", [8, 504, 512, 520, 1032])
def test_conv_channels(C):
    check_conv(conv_case(C, [5, 90, 2], C, 4, True, True), [5, 90, 2])


def test_conv_long_rows_and_many_sequences():
    lengths = [700, 1, 0, 3000, 2] + [3] * 400
    check_conv(conv_case(3, lengths, 40, 4, True, True), lengths)
    check_conv(conv_case(4, [1] * 300, 520, 4, True, True), [1] * 300, cu=False)


@pytest.mark.parametrize("C", [24, 520])
def test_conv_runs_of_empty_sequences(C):
    lengths = [0] * 700 + [5] + [0] * 2000 + [40, 0, 1] + [0] * 90 + [2] + [0] * 33 + [66] + [0] * 500
    check_conv(conv_case(10, lengths, C, 4, True, True), lengths)


def test_conv_wide_rows_go_by_the_longer_strips():
    check_conv(conv_case(5, [4000, 100], 8 * 640, 4, False, True), [4000, 100])


def test_conv_strided_rows_and_in_place_state():
    lengths = [1, 70, 2, 0, 5]
    x, w, b, init = conv_case(6, lengths, 64, 4, True, True)
    wide = torch.zeros(sum(lengths), 64 + 40, dtype=torch.bfloat16)
    wide[:, 8:72] = x
    want, tol, state = ref.conv(x, w, b, init, lengths, True)
    held = init.cuda()
    out, fin = kda.kda_conv_fwd(wide.cuda()[:, 8:72], w.cuda(), b.cuda(), initial_state=held, cu_seqlens=cu_of(lengths).cuda(),
                                final_state=held)
    ok()
    within(out, want, tol, "out")
    assert fin.data_ptr() == held.data_ptr() and torch.equal(held.double().cpu(), state)


def test_conv_extremes():
    lengths = [40]
    x, w, b, init = conv_case(7, lengths, 16, 4, True, True, amp=200.0)   # e^{-y} over- and underflows
    check_conv((x, w, b, init), lengths)
    x[20, 3] = float("nan")
    out, _ = kda.kda_conv_fwd(x.cuda(), w.cuda(), b.cuda(), initial_state=init.cuda())
    bad = torch.isnan(out).cpu()
    assert bad[20:24, 3].all() and bad.sum() == 4


def test_conv_rows_behind_the_last_sequence_stay():
    lengths = [5, 3]
    x, w, b, init = conv_case(8, [20], 16, 4, False, False)
    out = torch.full((20, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_conv_fwd(x.cuda(), w.cuda(), cu_seqlens=cu_of(lengths).cuda(), out=out)
    ok()
    want, tol, _ = ref.conv(x[:8], w, None, None, lengths, True)
    within(out[:8], want, tol, "out")
    assert (out[8:] == 7).all()


def test_conv_in_pieces_is_one_pass():
    x, w, b, _ = conv_case(9, [50], 32, 4, True, False)
    whole, last = kda.kda_conv_fwd(x.cuda(), w.cuda(), b.cuda())
    state, parts = None, []
    for r in (slice(0, 1), slice(1, 3), slice(3, 3), slice(3, 40), slice(40, 50)):
        o, state = kda.kda_conv_fwd(x[r].cuda(), w.cuda(), b.cuda(), initial_state=state)
        parts.append(o)
    ok()
    assert torch.equal(torch.cat(parts), whole) and torch.equal(state, last)


# ------------------------------------------------------------------ state-space recurrence

def ssm_case(seed, lengths, H, G, P, S, state="fp32", skip=True, bias=True, rate=4.0, step=1.0):
    g = gen(seed)
    T = sum(lengths)
    x, B, C = randn(g, T, H, P), randn(g, T, G, S), randn(g, T, G, S)
    dt = (step * torch.randn((T, H), generator=g) - 1.0).to(torch.bfloat16)
    A = -rate * torch.rand(H, generator=g)
    sk = torch.randn(H, generator=g) if skip else None
    db = torch.randn(H, generator=g) if bias else None
    init = None
    if state:
        init = torch.randn((len(lengths), H, P, S), generator=g)
        init = init.to(torch.bfloat16) if state == "bf16" else init
    return x, dt, A, B, C, sk, db, init


def run_ssm(entry, case, lengths, cu=True, **kw):
    *a, init = [dev(t) for t in case]
    kw.setdefault("initial_state", init)
    r = getattr(kda, entry)(*a, cu_seqlens=cu_of(lengths).cuda() if cu else None, N=None if cu else len(lengths), **kw)
    ok()
    return r


def check_ssm(entry, case, lengths, cu=True, final=True, **kw):
    out, fin = run_ssm(entry, case, lengths, cu, **({} if final else dict(output_final_state=False)), **kw)
    dtype = fin.dtype if final else torch.float32
    if entry == "kda_ssm_step":
        want, tol, state, stol = ref.ssm_step(*case, lengths, dtype)
    else:
        want, tol, state, stol = ref.ssm_chunks(*case, lengths, dtype, final)
    within(out, want, tol, "out")
    assert (fin is None) == (not final)
    if final:
        within(fin, state, stol, "state")
    return out, fin


HEADS = [(2, 1, 64, 128), (1, 1, 64, 128), (3, 1, 64, 64), (6, 2, 64, 128), (10, 2, 64, 64), (2, 2, 128, 64), (1, 1, 128, 128),
         (3, 1, 128, 128)]


@pytest.mark.parametrize("H,G,P,S", HEADS)
@pytest.mark.parametrize("state", ["fp32", "bf16", None])
def test_step(H, G, P, S, state):
    lengths = [1, 0, 3, 1, 8]
    check_ssm("kda_ssm_step", ssm_case(H + P + S, lengths, H, G, P, S, state), lengths)


@pytest.mark.parametrize("lengths", [[1], [2, 0, 1], [16], [127], [128], [129], [64, 65], [255, 1, 0, 257], [600], [0, 0], [385, 513, 33]])
@pytest.mark.parametrize("state", ["fp32", "bf16", None])
def test_fwd(lengths, state):
    check_ssm("kda_ssm_fwd", ssm_case(len(lengths) + sum(lengths), lengths, 2, 1, 64, 128, state), lengths)


@pytest.mark.parametrize("H,G,P,S", HEADS)
@pytest.mark.parametrize("state", ["fp32", "bf16"])
def test_fwd_heads(H, G, P, S, state):
    lengths = [130, 7]
    check_ssm("kda_ssm_fwd", ssm_case(7 * H + G + P + S, lengths, H, G, P, S, state), lengths)


@pytest.mark.parametrize("entry", ["kda_ssm_fwd", "kda_ssm_step"])
@pytest.mark.parametrize("skip,bias,state,final", [(False, False, "fp32", True), (True, False, None, False), (False, True, "fp32", False)])
def test_options(entry, skip, bias, state, final):
    lengths = [140, 20]
    check_ssm(entry, ssm_case(11, lengths, 4, 2, 64, 64, state, skip, bias), lengths, final=final)


# few sequences: cut into pieces that are joined through their states
@pytest.mark.parametrize("lengths,H,G,P,S,state", [
    ([3000], 2, 1, 64, 128, "fp32"), ([1500, 10, 0, 2200], 3, 1, 64, 64, "bf16"), ([2048], 1, 1, 128, 64, None),
    ([1023, 1025], 2, 2, 64, 128, "fp32"), ([4100], 1, 1, 128, 128, "fp32")])
def test_pieces(lengths, H, G, P, S, state):
    assert kda.kda_ssm_workspace_size(sum(lengths), H, G, len(lengths), P, S) > 0
    case = ssm_case(sum(lengths), lengths, H, G, P, S, state, rate=0.3, step=0.5)
    out, fin = check_ssm("kda_ssm_fwd", case, lengths)
    ws = torch.empty(kda.kda_ssm_workspace_size(sum(lengths), H, G, len(lengths), P, S), dtype=torch.uint8, device="cuda")
    again, fin2 = run_ssm("kda_ssm_fwd", case, lengths, workspace=ws.fill_(255))
    assert torch.equal(out, again) and torch.equal(fin, fin2)
    if state:  # in place
        held = case[-1].cuda()
        once, fin3 = run_ssm("kda_ssm_fwd", case, lengths, initial_state=held, final_state=held)
        assert fin3.data_ptr() == held.data_ptr() and torch.equal(once, out) and torch.equal(held, fin)


def test_whole_sequences_in_the_order_of_their_lengths():
    g = gen(5)
    lengths = torch.randint(0, 300, (90,), generator=g).tolist()
    assert kda.kda_ssm_workspace_size(sum(lengths), 4, 1, 90, 64, 64) == 0
    check_ssm("kda_ssm_fwd", ssm_case(12, lengths, 4, 1, 64, 64), lengths)
    lengths = [40] * 300                      # more than are ordered
    check_ssm("kda_ssm_fwd", ssm_case(13, lengths, 2, 1, 64, 64), lengths)
    check_ssm("kda_ssm_fwd", ssm_case(14, [100] * 80, 4, 1, 64, 64), [100] * 80, cu=False)


@pytest.mark.parametrize("entry", ["kda_ssm_fwd", "kda_ssm_step"])
def test_strided_rows_and_in_place_states(entry):
    lengths, H, G, P, S = [150, 0, 33, 1], 4, 2, 64, 128
    x, dt, A, B, C, sk, db, init = case = ssm_case(15, lengths, H, G, P, S)
    T = sum(lengths)
    rows = torch.cat([x.reshape(T, -1), B.reshape(T, -1), C.reshape(T, -1), randn(gen(1), T, 24)], 1).cuda()
    steps = torch.cat([dt, dt, dt[:, :1]], 1).cuda()[:, 1 + H - 1:2 * H]
    n = H * P
    held = init.cuda()
    out, fin = getattr(kda, entry)(rows[:, :n].view(T, H, P), steps, A.cuda(), rows[:, n:n + G * S].view(T, G, S),
                                   rows[:, n + G * S:n + 2 * G * S].view(T, G, S), sk.cuda(), db.cuda(), initial_state=held,
                                   cu_seqlens=cu_of(lengths).cuda(), final_state=held)
    ok()
    plain, state = run_ssm(entry, case, lengths)
    assert torch.equal(out, plain) and torch.equal(fin, state) and fin.data_ptr() == held.data_ptr()


@pytest.mark.parametrize("entry", ["kda_ssm_fwd", "kda_ssm_step"])
@pytest.mark.parametrize("rate,step", [(60.0, 30.0), (1e-4, 0.1), (0.0, 1.0)])
def test_decays_strong_and_none(entry, rate, step):
    lengths = [300, 128]
    check_ssm(entry, ssm_case(16, lengths, 2, 1, 64, 128, rate=rate, step=step), lengths)


@pytest.mark.parametrize("entry", ["kda_ssm_fwd", "kda_ssm_step"])
def test_other_sequences_rows_do_not_show(entry):
    lengths = [37, 100, 128, 60]
    case = ssm_case(17, lengths, 3, 1, 64, 128)
    out, fin = run_ssm(entry, case, lengths)
    spoilt = [t.clone() for t in case]
    for i in (0, 1, 3, 4):
        spoilt[i][137:265] = float("nan")   # all of the third sequence
    spoilt[7][2] = float("inf")
    got, state = run_ssm(entry, spoilt, lengths)
    keep = [0, 1, 3]
    assert torch.equal(torch.cat([got[:137], got[265:]]), torch.cat([out[:137], out[265:]]))
    assert torch.equal(state[keep], fin[keep])


@pytest.mark.parametrize("entry", ["kda_ssm_fwd", "kda_ssm_step"])
def test_rows_behind_the_last_sequence_stay(entry):
    lengths = [130, 5]
    case = ssm_case(18, [200], 2, 1, 64, 64, state=None)
    out = torch.full((200, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    run_ssm(entry, case, lengths, out=out)
    assert (out[135:] == 3).all()
    short = [t[:135] if t is not None and t.shape[0] == 200 else t for t in case]
    assert torch.equal(out[:135], run_ssm(entry, short, lengths)[0])


def test_a_sequence_in_parts_is_one_pass():
    """A prompt, then tokens one at a time: the state carries on between the two schedules."""
    T = 260
    case = ssm_case(19, [T], 2, 1, 64, 128, rate=1.0)
    x, dt, A, B, C, sk, db, init = case
    want, tol, state, stol = ref.ssm_step(*case, [T])
    chunk, ctol, cstate, cstol = ref.ssm_chunks(*[t[:256] if t.shape[0] == T else t for t in case], [256])
    cut = lambda r: [dev(t[r]) if t.shape[0] == T else dev(t) for t in (x, dt, A, B, C, sk, db)]  # noqa: E731
    o, m = kda.kda_ssm_fwd(*cut(slice(0, 256)), initial_state=init.cuda())
    within(o, chunk, ctol, "prompt")
    for t in range(256, T):
        o, m = kda.kda_ssm_step(*cut(slice(t, t + 1)), initial_state=m, final_state=m)
        # what the prompt's state is off by decays or stays
        within(o, want[t:t + 1], tol[t:t + 1] + torch.einsum("hps,hs->hp", cstol[0], C[t].double().abs().expand(2, -1)), "token")
    ok()
    within(m, state, stol + cstol, "state")


@pytest.mark.parametrize("bad", [[0, 50, 30, 100], [-5, 20, 400, 100], [90, 80, 70, 60], [0, 0, 1 << 30, -(1 << 30)]])
def test_malformed_cu_seqlens_stay_in_bounds(bad):
    case = ssm_case(20, [100], 2, 1, 64, 64, state=None)
    guard = torch.full((120, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
    *a, _ = [dev(t) for t in case]
    for entry in ("kda_ssm_fwd", "kda_ssm_step"):
        _, fin = getattr(kda, entry)(*a, cu_seqlens=cu, out=guard[:100])
        assert fin.shape == (3, 2, 64, 64)
    x, w, _, _ = conv_case(1, [100], 32, 4, False, False)
    out = torch.full((120, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_conv_fwd(x.cuda(), w.cuda(), cu_seqlens=cu, out=out[:100])
    ok()
    assert (guard[100:] == 5).all() and (out[100:] == 5).all()


# ------------------------------------------------------------------ streams, graphs, refusals

def test_two_streams_at_once():
    lengths = [2500]
    cases = [ssm_case(30 + i, lengths, 2, 1, 64, 128, rate=0.5) for i in range(4)]
    want = [run_ssm("kda_ssm_fwd", c, lengths) for c in cases]
    args = [[dev(t) for t in c] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(3):
        got.append([kda.kda_ssm_fwd(*a[:-1], initial_state=a[-1], cu_seqlens=cu_of(lengths).cuda(), stream=s)
                    for a, s in zip(args, streams)])
    torch.cuda.synchronize()
    ok()
    for row in got:
        for (o, m), (ow, mw) in zip(row, want):
            assert torch.equal(o, ow) and torch.equal(m, mw)


@pytest.mark.parametrize("lengths", [[2100], [200, 70, 1]])
def test_captured_into_graphs_that_share_a_workspace(lengths):
    H, G, P, S = 2, 1, 64, 128
    cases = [ssm_case(40 + i, lengths, H, G, P, S, rate=0.5) for i in range(2)]
    want = [run_ssm("kda_ssm_fwd", c, lengths) for c in cases]
    size = max(1, kda.kda_ssm_workspace_size(sum(lengths), H, G, len(lengths), P, S))
    ws, cu = torch.empty(size, dtype=torch.uint8, device="cuda"), cu_of(lengths).cuda()
    graphs, outs = [], []
    args = [[dev(t) for t in c] for c in cases]
    torch.cuda.synchronize()
    for a in args:
        held = a[-1].clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(kda.kda_ssm_fwd(*a[:-1], initial_state=a[-1], cu_seqlens=cu, final_state=held, workspace=ws))
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        ok()
        for (o, m), (ow, mw) in zip(outs, want):
            assert torch.equal(o, ow) and torch.equal(m, mw)
            o.zero_(), m.zero_()


def test_a_captured_step_of_both():
    """The convolution and the step of one token, states in place, replayed."""
    N, H, G, P, S = 5, 2, 1, 64, 64
    C = H * P + 2 * G * S
    g = gen(50)
    x, w = randn(g, N, C).cuda(), randn(g, C, 4).cuda()
    dt, A = randn(g, N, H).cuda(), (-torch.rand(H, generator=g)).cuda()
    first = randn(g, N, 3, C).cuda(), torch.randn((N, H, P, S), generator=g).cuda()

    def step(conv, m):
        rows, _ = kda.kda_conv_fwd(x, w, initial_state=conv, N=N, final_state=conv)
        n = H * P
        return kda.kda_ssm_step(rows[:, :n].view(N, H, P), dt, A, rows[:, n:n + G * S].view(N, G, S),
                                rows[:, n + G * S:].view(N, G, S), initial_state=m, N=N, final_state=m)[0]

    conv, m = first[0].clone(), first[1].clone()
    want = [step(conv, m).clone() for _ in range(3)]
    last = conv.clone(), m.clone()
    conv, m = first[0].clone(), first[1].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(conv, m)
    conv.copy_(first[0]), m.copy_(first[1])
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k])
    ok()
    assert torch.equal(conv, last[0]) and torch.equal(m, last[1])


def test_refusals():
    x, dt, A, B, C, sk, db, init = [dev(t) for t in ssm_case(60, [20], 2, 1, 64, 64)]
    for entry in (kda.kda_ssm_fwd, kda.kda_ssm_step):
        with pytest.raises(TypeError, match="float32"):
            entry(x, dt, A.half(), B, C)
        with pytest.raises(TypeError, match="float32 or torch.bfloat16"):
            entry(x, dt, A, B, C, initial_state=init.half())
        with pytest.raises(TypeError, match="final_state must be torch.float32"):
            entry(x, dt, A, B, C, initial_state=init, final_state=init.bfloat16())
        with pytest.raises(ValueError, match="shape"):
            entry(x, dt, A, B, C[:, :, :32])
        with pytest.raises(ValueError, match="contiguous"):
            entry(x.transpose(0, 1).contiguous().transpose(0, 1), dt, A, B, C)
        with pytest.raises(ValueError, match="elements apart"):
            entry(x[:1].expand(20, 2, 64), dt, A, B, C)
        with pytest.raises(ValueError, match="contiguous"):
            entry(x, dt, A, B, C, skip=torch.zeros(4, device="cuda")[::2])
        with pytest.raises(ValueError, match="N is 2"):
            entry(x, dt, A, B, C, cu_seqlens=cu_of([20]).cuda(), N=2)
        with pytest.raises(kda.KdaError, match="INVALID_ARG"):
            entry(x, dt, A, B, C, out=x)
    rows, w = torch.zeros(6, 24, device="cuda").bfloat16(), torch.zeros(24, 4, device="cuda").bfloat16()
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):
        kda.kda_conv_fwd(rows, w, out=rows)
    with pytest.raises(kda.KdaError, match="UNSUPPORTED"):
        kda.kda_conv_fwd(rows, torch.zeros(24, 5, device="cuda").bfloat16())
    with pytest.raises(ValueError, match="elements apart"):
        kda.kda_conv_fwd(torch.zeros(6, 25, device="cuda").bfloat16()[:, :24], w)
    with pytest.raises(TypeError, match="bfloat16"):
        kda.kda_conv_fwd(rows, w, initial_state=torch.zeros(1, 3, 24, device="cuda"))
    ok()


def test_the_layer_serves_a_prompt_and_its_continuation():
    """The example's path: prompts, then tokens one at a time, against one pass over all of them."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import state_space_layer
    report = state_space_layer.main(["--tokens", "300", "--steps", "5", "--heads", "6"])
    # the outputs of both are rounded to bf16 at the end and a few times on the way
    assert report["outputs_differ"] < 1e-2 and report["states_differ"] < 1e-4
