"""Attention over packed rows, the 8-bit cache, attention over it and eviction
on the GPU against the 64-bit forms of attn_ref."""
import itertools
import random

import pytest
import torch

import attn_ref as ref
import chunked_gated_delta_11_gb300 as kda

pytestmark = pytest.mark.gpu

D = 128
SCALE = D ** -0.5


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


# ------------------------------------------------------------------ packed rows

def prefill_case(seed, lengths, H, Hk, mask, cap, bias, amp=2.0):
    g = gen(seed)
    T = sum(lengths)
    q, k, v = amp * randn(g, T, H, D), randn(g, T, Hk, D), randn(g, T, Hk, D)
    slopes = 0.5 * torch.rand(H, generator=g) if bias else None
    prefix = None
    if mask == "prefix":
        prefix = torch.tensor([random.Random(seed + i).choice([0, n // 3, n // 2, n, n + 7, -2])
                               for i, n in enumerate(lengths)], dtype=torch.int32)
    return q, k, v, slopes, prefix


def run_prefill(q, k, v, lengths, mask, cap, slopes, prefix, cu=True, **kw):
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    return kda.kda_attn_fwd(dev(q), dev(k), dev(v), SCALE, mask=mask, cap=cap, slopes=dev(slopes),
                            prefix_lens=dev(prefix), cu_seqlens=cu_of(lengths).cuda() if cu else None,
                            N=None if cu else len(lengths), **kw)


@pytest.mark.parametrize("lengths", [[1], [2, 0, 1], [64], [127, 128], [129], [255, 1, 0, 257], [600], [385, 513]])
@pytest.mark.parametrize("mask", ["causal", "full", "prefix"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (5.0, True)])
def test_prefill(lengths, mask, cap, bias):
    q, k, v, slopes, prefix = prefill_case(len(lengths) + sum(lengths), lengths, 4, 2, mask, cap, bias)
    out = run_prefill(q, k, v, lengths, mask, cap, slopes, prefix)
    ok()
    want, tol = ref.prefill(q, k, v, SCALE, lengths, mask, cap, slopes, prefix)
    within(out, want, tol, "out")


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (6, 6), (16, 2), (5, 5)])
def test_prefill_heads(H, Hk):
    lengths = [200, 77]
    q, k, v, _, _ = prefill_case(H, lengths, H, Hk, "causal", 0.0, False)
    want, tol = ref.prefill(q, k, v, SCALE, lengths, "causal")
    within(run_prefill(q, k, v, lengths, "causal", 0.0, None, None), want, tol, "out")
    ok()


def test_prefill_equal_sequences_without_cu_seqlens():
    lengths = [150] * 3
    q, k, v, _, _ = prefill_case(3, lengths, 2, 1, "full", 0.0, False)
    want, tol = ref.prefill(q, k, v, SCALE, lengths, "full")
    within(run_prefill(q, k, v, lengths, "full", 0.0, None, None, cu=False), want, tol, "out")
    ok()


@pytest.mark.parametrize("amp", [0.0, 30.0, 300.0])
def test_prefill_flat_and_peaked_scores(amp):
    lengths = [300]
    q, k, v, _, _ = prefill_case(9, lengths, 2, 2, "causal", 0.0, False, amp=amp)
    want, tol = ref.prefill(q, k, v, SCALE, lengths, "causal")
    within(run_prefill(q, k, v, lengths, "causal", 0.0, None, None), want, tol, "out")
    ok()


@pytest.mark.parametrize("slope", [-0.05, 40.0])
def test_prefill_rising_bias_and_one_that_leaves_only_the_token_itself(slope):
    lengths = [400]
    q, k, v, _, _ = prefill_case(10, lengths, 2, 1, "full", 0.0, False)
    slopes = torch.full((2,), slope)
    want, tol = ref.prefill(q, k, v, SCALE, lengths, "full", slopes=slopes)
    within(run_prefill(q, k, v, lengths, "full", 0.0, slopes, None), want, tol, "out")
    ok()


def test_prefill_ascending_scores_move_the_running_maximum():
    # every key scores higher than the ones before it
    n = 700
    q = torch.zeros((n, 1, D), dtype=torch.bfloat16)
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16)
    q[:, :, 0] = 16.0
    k[:, 0, 0] = (torch.arange(n) * 0.5).to(torch.bfloat16)
    v = randn(gen(1), n, 1, D)
    want, tol = ref.prefill(q, k, v, SCALE, [n], "full")
    within(run_prefill(q, k, v, [n], "full", 0.0, None, None), want, tol, "out")
    ok()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("mask", ["causal", "full"])
def test_prefill_other_sequences_reach_no_result(bad, mask):
    lengths = [130, 70, 300]
    q, k, v, _, _ = prefill_case(4, lengths, 2, 1, mask, 0.0, False)
    want, tol = ref.prefill(q, k, v, SCALE, lengths, mask)
    for x in (q, k, v):
        x[130:200] = bad
    out = run_prefill(q, k, v, lengths, mask, 0.0, None, None)
    ok()
    for rows in (slice(0, 130), slice(200, 500)):
        within(out[rows], want[rows], tol[rows], "out")


# more (256 rows, head) pieces of work than SMs, so that a CTA takes several
MANY = [random.Random(7).choice([0, 1, 17, 64, 128, 129, 250, 257, 300]) for _ in range(60)]


@pytest.mark.parametrize("lengths,H,Hk", [(MANY, 8, 2), ([900, 1300, 0, 20], 32, 4), ([40] * 200, 4, 4)],
                         ids=["ragged", "long", "short"])
@pytest.mark.parametrize("mask", ["causal", "full", "prefix"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (5.0, True)])
def test_prefill_more_work_than_sms(lengths, H, Hk, mask, cap, bias):
    q, k, v, slopes, prefix = prefill_case(21, lengths, H, Hk, mask, cap, bias)
    out = run_prefill(q, k, v, lengths, mask, cap, slopes, prefix)
    ok()
    want, tol = ref.prefill(q, k, v, SCALE, lengths, mask, cap, slopes, prefix)
    within(out, want, tol, "out")
    assert torch.equal(out, run_prefill(q, k, v, lengths, mask, cap, slopes, prefix))
    ok()


def test_prefill_more_work_than_sms_in_a_graph():
    q, k, v, _, _ = (x if x is None else x.cuda() for x in prefill_case(22, MANY, 8, 2, "causal", 0.0, False))
    cu, out = cu_of(MANY).cuda(), torch.empty_like(q)
    want = kda.kda_attn_fwd(q, k, v, SCALE, cu_seqlens=cu).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            kda.kda_attn_fwd(q, k, v, SCALE, cu_seqlens=cu, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    ok()


def test_prefill_malformed_cu_seqlens_with_more_work_than_sms():
    q, k, v, _, _ = prefill_case(6, [600], 64, 8, "causal", 0.0, False)
    pad = torch.full((632, 64, D), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([-5, 900, 30, 2000, 590, 600], dtype=torch.int32).cuda()
    kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), SCALE, cu_seqlens=cu, out=pad[16:616])
    torch.cuda.synchronize()
    assert (pad[:16] == 7).all() and (pad[616:] == 7).all()


@pytest.mark.parametrize("lengths,H,Hk", [([640], 2, 1), ([1100], 3, 1), ([2200], 2, 2), ([2047, 1, 2500], 1, 1),
                                          ([0, 1537], 2, 1)])
@pytest.mark.parametrize("mask", ["causal", "full", "prefix"])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, True)])
def test_prefill_few_pieces_shared_by_several_ctas(lengths, H, Hk, mask, cap, bias):
    q, k, v, slopes, prefix = prefill_case(31, lengths, H, Hk, mask, cap, bias)
    out = run_prefill(q, k, v, lengths, mask, cap, slopes, prefix)
    ok()
    want, tol = ref.prefill(q, k, v, SCALE, lengths, mask, cap, slopes, prefix)
    within(out, want, tol, "out")
    assert torch.equal(out, run_prefill(q, k, v, lengths, mask, cap, slopes, prefix))
    ok()


def test_prefill_shared_pieces_of_a_malformed_cu_seqlens():
    q, k, v, _, _ = prefill_case(32, [2000], 2, 1, "causal", 0.0, False)
    pad = torch.full((2032, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([-5, 3000, 30], dtype=torch.int32).cuda()
    kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), SCALE, cu_seqlens=cu, out=pad[16:2016])
    torch.cuda.synchronize()
    assert (pad[:16] == 7).all() and (pad[2016:] == 7).all()


def test_prefill_malformed_cu_seqlens_stays_in_bounds():
    q, k, v, _, _ = prefill_case(5, [64], 2, 1, "causal", 0.0, False)
    pad = torch.full((96, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([-5, 90, 30, 1000], dtype=torch.int32).cuda()
    kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), SCALE, cu_seqlens=cu, out=pad[16:80])
    torch.cuda.synchronize()
    assert (pad[:16] == 7).all() and (pad[80:] == 7).all()


def test_prefill_same_bits_and_other_streams_and_graphs():
    lengths = [500, 31]
    q, k, v, _, _ = prefill_case(6, lengths, 4, 2, "causal", 30.0, False)
    a = run_prefill(q, k, v, lengths, "causal", 30.0, None, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = run_prefill(q, k, v, lengths, "causal", 30.0, None, None, stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    qd, kd, vd, cu = q.cuda(), k.cuda(), v.cuda(), cu_of(lengths).cuda()
    out = torch.empty_like(qd)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kda.kda_attn_fwd(qd, kd, vd, SCALE, cap=30.0, cu_seqlens=cu, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out)
    ok()


def test_prefill_offsets_past_32_bits():
    T, H = 1_200_000, 16                       # 2.46e9 elements of q
    n = 50
    q = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda").normal_()
    k = torch.empty((T, 1, D), dtype=torch.bfloat16, device="cuda").normal_()
    v = torch.empty((T, 1, D), dtype=torch.bfloat16, device="cuda").normal_()
    out = kda.kda_attn_fwd(q, k, v, SCALE, N=T // n)
    ok()
    for a in (0, T - n):
        rows = slice(a, a + n)
        want, tol = ref.prefill(q[rows].cpu(), k[rows].cpu(), v[rows].cpu(), SCALE, [n], "causal")
        within(out[rows], want, tol, "out")


# ------------------------------------------------------------------ the cache

def table_of(lens, page, seed, spare=2, width_more=1):
    """Shuffled pages for these lengths: table (-1 past them) and the pool's size."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    perm = list(range(pages))
    random.Random(seed).shuffle(perm)
    width = max(1, max(need)) + width_more
    rows, at = [], 0
    for m in need:
        rows.append(perm[at:at + m] + [-1] * (width - m))
        at += m
    return torch.tensor(rows, dtype=torch.int32), pages


def filled(lens, Hk, page, seed, scale_spread=2):
    """A pool whose used slots hold values, and every other slot NaN codes and wild numbers."""
    g = gen(seed)
    table, pages = table_of(lens, page, seed)
    codes = [torch.randn((pages, Hk, page, D), generator=g).mul_(40).clamp_(-448, 448).to(torch.float8_e4m3fn)
             for _ in range(2)]
    scales = [torch.exp2(torch.randint(-5 - scale_spread, -4, (pages, Hk), generator=g).float()) for _ in range(2)]
    pos = torch.randint(-50, 50, (pages, Hk, page), generator=g, dtype=torch.int32)
    weight = torch.rand((pages, Hk, page), generator=g)
    nan = torch.tensor(0x7f, dtype=torch.uint8)
    used = torch.zeros((pages, page), dtype=torch.bool)
    for n, row in zip(lens, table):
        for j in range(-(-n // page)):
            m = min(page, n - j * page)
            used[int(row[j]), :m] = True
            pos[int(row[j]), :, :m] = torch.arange(j * page, j * page + m, dtype=torch.int32)
    hole = ~used[:, None, :, None].expand(-1, Hk, -1, D)
    for c in codes:
        c.view(torch.uint8)[hole] = nan
    return kda.KvCache(*codes, *scales, pos, weight), table


def to(cache, device):
    return kda.KvCache(*(t.to(device) for t in cache))


def check_cached(cache, table, lens, H, counts, seed, cap=0.0, bias=False, positions=None, weights=True, amp=2.0):
    g = gen(seed + 1)
    q = amp * randn(g, sum(counts), H, D)
    slopes = 0.2 * torch.rand(H, generator=g) if bias else None
    want, tol, add, addtol = ref.cached(cache, q, table, lens, SCALE, counts, cap, slopes, positions)
    dev = to(cache, "cuda")
    lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
    equal = len(set(counts)) == 1
    out = kda.kda_cache_attn(dev, q.cuda(), table.cuda(), lens_t, SCALE, cap=cap,
                             slopes=None if slopes is None else slopes.cuda(),
                             cu_seqlens=None if equal else cu_of(counts).cuda(),
                             positions=None if positions is None else positions.cuda(), accumulate=weights)
    ok()
    within(out, want, tol, "out")
    if weights:
        was = cache.weight.double()
        within(dev.weight, was + add, addtol + 4 * ref.F32 * (was + add), "weight")
        same = add == 0
        assert torch.equal(dev.weight.cpu()[same], cache.weight[same])
    for a, b in zip(dev[:5], cache[:5]):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
    return out


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 1), (8, 1), (12, 1), (16, 1), (6, 2), (34, 1), (8, 8)])
def test_cached_single_tokens(page, H, Hk):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 129, 300]
    cache, table = filled(lens, Hk, page, page + H)
    check_cached(cache, table, lens, H, [1] * len(lens), page * H)


@pytest.mark.parametrize("cap,bias", [(20.0, False), (0.0, True), (3.0, True)])
@pytest.mark.parametrize("page", [16, 64])
def test_cached_scores(page, cap, bias):
    lens = [200, 1, 33, 700]
    cache, table = filled(lens, 2, page, 5)
    check_cached(cache, table, lens, 8, [1] * 4, 6, cap, bias)


@pytest.mark.parametrize("H,Hk", [(1, 1), (8, 2), (16, 1), (10, 2)])
@pytest.mark.parametrize("counts", [[4, 4, 4], [1, 5, 2], [0, 9, 3], [30, 1, 17]])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (10.0, True)])
def test_cached_several_tokens(H, Hk, counts, cap, bias):
    lens = [40, 300, 77]
    cache, table = filled(lens, Hk, 32, 7)
    check_cached(cache, table, lens, H, counts, 8, cap, bias)


def test_cached_queries_alone_and_before_everything():
    # a prompt of its own in the cache, and more queries than slots
    cache, table = filled([8, 3], 2, 16, 11)
    check_cached(cache, table, [8, 3], 4, [8, 5], 12)


def test_cached_positions_with_gaps():
    """Positions as eviction leaves them, queries at given ones: some see nothing."""
    lens = [150, 90]
    cache, table = filled(lens, 2, 16, 13)
    for row, n in zip(table, lens):
        slots = sorted(random.Random(n).sample(range(10, 4000), n))
        for j in range(-(-n // 16)):
            m = min(16, n - 16 * j)
            cache.pos[int(row[j]), :, :m] = torch.tensor(slots[16 * j:16 * j + m], dtype=torch.int32)
    positions = torch.tensor([5, 2000, 4000, 11, 3999, 700], dtype=torch.int32)
    check_cached(cache, table, lens, 8, [3, 3], 14, bias=True, positions=positions)
    check_cached(cache, table, lens, 8, [3, 3], 14)


@pytest.mark.parametrize("lens", [[5000], [4096, 1, 2500], [20000, 30]])
@pytest.mark.parametrize("H,Hk,counts", [(8, 1, 1), (4, 2, 1), (16, 1, 3)])
def test_cached_long_sequences(lens, H, Hk, counts):
    cache, table = filled(lens, Hk, 64, sum(lens))
    check_cached(cache, table, lens, H, [counts] * len(lens), 15, bias=True)


@pytest.mark.parametrize("H", [24, 64])
def test_cached_weights_of_many_slots_and_rows(H):
    lens = [12000, 9000, 100, 11000]  # enough slots for the weight sums to fill the GPU
    cache, table = filled(lens, 4, 64, H)
    check_cached(cache, table, lens, H, [2] * 4, 19)


@pytest.mark.parametrize("amp", [0.0, 60.0])
def test_cached_flat_and_peaked_scores_and_far_scales(amp):
    lens = [900, 64]
    cache, table = filled(lens, 2, 32, 16, scale_spread=16)
    check_cached(cache, table, lens, 6, [1, 1], 17, amp=amp)


def test_cached_large_and_tiny_queries():
    lens = [100]
    cache, table = filled(lens, 1, 16, 18)
    for amp in (2.0 ** -30, 2.0 ** 20):
        small = cache._replace(k_scale=cache.k_scale / amp)
        check_cached(small, table, lens, 4, [1], 19, amp=amp)


def test_cached_wide_table_and_same_bits():
    """Many more table columns than the sequences need; two calls give the same bits."""
    lens = [3000, 10, 700]
    cache, table = filled(lens, 1, 16, 20)
    wide = torch.full((3, 5000), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    a = check_cached(cache, wide, lens, 8, [1] * 3, 21)
    b = check_cached(cache, wide, lens, 8, [1] * 3, 21)
    assert torch.equal(a, b)


@pytest.mark.parametrize("H,Hk,counts", [(8, 8, 1), (12, 4, 1), (16, 2, None), (32, 2, 3)])
@pytest.mark.parametrize("bias", [False, True])
def test_cached_many_short_sequences_in_a_very_wide_table(H, Hk, counts, bias):
    """The grid of all possible chunks would be mostly empty: a list of the real ones is used."""
    r = random.Random(H)
    lens = [r.choice([0, 1, 3, 16, 20, 40]) for _ in range(699)] + [5000]
    cache, table = filled(lens, Hk, 16, 24 + H)
    wide = torch.full((700, 4000), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    each = [counts] * 700 if counts else [r.choice([0, 1, 2, 5]) for _ in range(700)]
    check_cached(cache, wide, lens, H, each, 25, bias=bias)


@pytest.mark.parametrize("H,Hk", [(4, 4), (32, 2)])
def test_cached_malformed_cu_seqlens_stays_in_bounds(H, Hk):
    lens = [100, 50, 7, 300]
    cache, table = filled(lens, Hk, 16, 26)
    wide = torch.full((4, 4000), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    q = randn(gen(5), 40, H, D).cuda()
    pad = torch.full((60, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    for tab in (table, wide):
        for cu in ([0, 40, 0, 40, 40], [-3, 100, 7, 2, 1 << 30]):
            kda.kda_cache_attn(to(cache, "cuda"), q, tab.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), SCALE,
                               cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), accumulate=True, out=pad[10:50])
            torch.cuda.synchronize()
            assert (pad[:10] == 7).all() and (pad[50:] == 7).all()
    ok()


def test_cached_streams_graphs_and_own_workspace():
    lens = [900, 33]
    cache, table = filled(lens, 2, 64, 22)
    q = randn(gen(3), 2, 8, D).cuda()
    lens_t, tab = torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda()

    def call(c, **kw):
        return kda.kda_cache_attn(c, q, tab, lens_t, SCALE, accumulate=True, **kw)

    c0 = to(cache, "cuda")
    a = call(c0)
    c1 = to(cache, "cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = call(c1, stream=s)
    s.synchronize()
    assert torch.equal(a, b) and torch.equal(c0.weight, c1.weight)
    c2, out = to(cache, "cuda"), torch.empty_like(q)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(c2, out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out) and torch.equal(c0.weight, c2.weight)
    ok()


def test_cached_bad_pages_and_lengths_are_reported_and_skipped():
    lens = [100, 50]
    cache, table = filled(lens, 1, 16, 23)
    q = randn(gen(4), 2, 4, D)
    for change in ("page", "negative", "length"):
        tab, n = table.clone(), list(lens)
        if change == "length":
            n[0] = 100_000
            tab[0] = torch.where(tab[0] < 0, tab[1, 0], tab[0])  # every column holds some page
            cache.pos.clamp_(min=0)
            cache.k.view(torch.uint8)[cache.k.view(torch.uint8) == 0x7f] = 0
            cache.v.view(torch.uint8)[cache.v.view(torch.uint8) == 0x7f] = 0
        else:
            tab[0, 2] = 1 << 20 if change == "page" else -7
        out = kda.kda_cache_attn(to(cache, "cuda"), q.cuda(), tab.cuda(),
                                 torch.tensor(n, dtype=torch.int32).cuda(), SCALE,
                                 positions=torch.tensor([99, 49], dtype=torch.int32).cuda())
        assert kda.kda_device_status() == 1, change
        want, tol, _, _ = ref.cached(cache, q, table, lens, SCALE, [1, 1],
                                     positions=torch.tensor([99, 49], dtype=torch.int32))
        within(out[1], want[1], tol[1], change)
        assert torch.isfinite(out).all()


def test_cached_offsets_past_32_bits():
    pages, Hk, page = 33_000, 8, 64                 # 2.16e9 codes
    c = kda.kda_cache_alloc(pages, Hk, page)
    lens = [300, 64]
    table = torch.full((2, 5), -1, dtype=torch.int32)
    ids = list(range(pages - 6, pages))
    table[0], table[1, 0] = torch.tensor(ids[:5], dtype=torch.int32), ids[5]
    k, v = randn(gen(5), 364, Hk, D), randn(gen(6), 364, Hk, D)
    zero = torch.zeros(2, dtype=torch.int32).cuda()
    kda.kda_cache_append(c, k.cuda(), v.cuda(), table.cuda(), zero, cu_seqlens=cu_of(lens).cuda())
    ok()
    part = kda.KvCache(*(t[pages - 6:].cpu() for t in c))
    near = torch.where(table >= 0, table - (pages - 6), -1)
    q = randn(gen(7), 2, 16, D)
    out = kda.kda_cache_attn(c, q.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), SCALE,
                             accumulate=True)
    ok()
    want, tol, add, addtol = ref.cached(part, q, near, lens, SCALE, [1, 1])
    within(out, want, tol, "out")
    within(c.weight[pages - 6:], add, addtol + 4 * ref.F32 * add, "weight")
    assert (c.weight[: pages - 6] == 0).all()


# ------------------------------------------------------------------ append

def as_values(cache):
    return {"k": cache.k.double(), "v": cache.v.double(), "k_scale": cache.k_scale.double(),
            "v_scale": cache.v_scale.double(), "pos": cache.pos.long(), "weight": cache.weight.double()}


def same_cache(got, want):
    for name, x in want.items():
        y = getattr(got, name).cpu().double()
        x = x.double()
        assert torch.equal(torch.isnan(x), torch.isnan(y)), name
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y)), name


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("lens,counts", [([0], [1]), ([0, 3, 0], [5, 0, 1]), ([15, 16, 17], [1, 1, 1]),
                                         ([0, 100, 63], [200, 1, 129]), ([127, 1], [130, 64])])
def test_append(page, lens, counts):
    g = gen(page + sum(counts))
    total = [a + b for a, b in zip(lens, counts)]
    table, pages = table_of(total, page, page)
    Hk, T = 3, sum(counts)
    cache, _ = filled([0], Hk, page, 1)
    n = cache.k.shape[0]
    grow = lambda x: x.repeat(-(-pages // n), *[1] * (x.dim() - 1))[:pages].contiguous()  # noqa: E731
    cache = kda.KvCache(*(grow(t.view(torch.uint8)).view(t.dtype) if t.dtype == torch.float8_e4m3fn else grow(t)
                          for t in cache))
    first = sum(lens)
    want = as_values(cache)
    dev = to(cache, "cuda")
    for have, cnt, rows in (([0] * len(lens), lens, first), (lens, counts, T)):
        size = torch.exp(2 * torch.randn((rows, Hk, 1), generator=g))
        k = (torch.randn((rows, Hk, D), generator=g) * size).to(torch.bfloat16)
        v = (torch.randn((rows, Hk, D), generator=g) * 1e-3 * size).to(torch.bfloat16)
        if rows > 3:
            k[1, 0, 5], v[2, 1, 7], v[3, 2, 0], k[0] = float("nan"), float("inf"), -float("inf"), 0.0
        kda.kda_cache_append(dev, k.cuda(), v.cuda(), table.cuda(), torch.tensor(have, dtype=torch.int32).cuda(),
                             cu_seqlens=cu_of(cnt).cuda())
        ref.append(want, k, v, table, have, cnt)
    ok()
    same_cache(dev, want)


def test_append_extreme_values_and_borders():
    edge = torch.tensor([448.0, 450.0, 1.75, 1.7578125, 2.0 ** -130, 3.3e38, -3.3e38, 0.0, 2.0 ** -56, 2.0 ** -57])
    k = edge.to(torch.bfloat16)[:, None, None].repeat(1, 1, D).contiguous()
    v = (-k.float() * 0.5).to(torch.bfloat16)
    table = torch.arange(10, dtype=torch.int32)[:, None].contiguous()
    dev = kda.kda_cache_alloc(10, 1, 16)
    want = as_values(to(dev, "cpu"))
    zero = torch.zeros(10, dtype=torch.int32)
    kda.kda_cache_append(dev, k.cuda(), v.cuda(), table.cuda(), zero.cuda())
    ref.append(want, k, v, table, [0] * 10, [1] * 10)
    ok()
    same_cache(dev, want)


def test_append_token_by_token_with_positions():
    dev = kda.kda_cache_alloc(4, 2, 16)
    want = as_values(to(dev, "cpu"))
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32)
    g = gen(2)
    for i in range(40):
        k, v = (2.0 ** (i % 7)) * randn(g, 1, 2, D), randn(g, 1, 2, D)
        positions = torch.tensor([3 * i + 1], dtype=torch.int32)
        kda.kda_cache_append(dev, k.cuda(), v.cuda(), table.cuda(), torch.tensor([i], dtype=torch.int32).cuda(),
                             positions=positions.cuda())
        ref.append(want, k, v, table, [i], [1], positions)
    ok()
    same_cache(dev, want)


def test_append_past_the_table_and_to_bad_pages_is_reported():
    k = randn(gen(1), 40, 1, D).cuda()
    for table, lens in ((torch.tensor([[1, 2]]), 0), (torch.tensor([[1, 9, 2]]), 0), (torch.tensor([[1, -1, 2]]), 0),
                        (torch.tensor([[0, 1, 2]]), -4)):
        dev = kda.kda_cache_alloc(4, 1, 16)
        kda.kda_cache_append(dev, k, k, table.int().cuda(), torch.tensor([lens], dtype=torch.int32).cuda())
        assert kda.kda_device_status() == 1
        assert (dev.k.view(torch.uint8)[3] == 0).all()


# ------------------------------------------------------------------ evict

@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("lens,budget,recent", [([100], 100, 10), ([0, 1, 40], 20, 20), ([300, 5, 129, 64], 64, 16),
                                                ([2500, 700], 130, 1), ([1500], 1000, 0), ([3000], 1, 1)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict(page, lens, budget, recent, ties):
    Hk = 2
    cache, table = filled(lens, Hk, page, sum(lens) + page)
    w = torch.randint(0, 3, cache.weight.shape, generator=gen(1)).float() if ties else \
        torch.exp(2 * torch.randn(cache.weight.shape, generator=gen(2)))
    w[w < 0.02] = -0.0
    kept = [min(n, budget) for n in lens]
    dst_rel, extra = table_of(kept, page, 3, spare=0)
    base = cache.k.shape[0]
    dst = torch.where(dst_rel >= 0, dst_rel + base, -1)
    more = lambda x: torch.cat([x, x[:1].expand(extra, *x.shape[1:])]) if extra else x  # noqa: E731
    cache = cache._replace(weight=w)
    cache = kda.KvCache(*(more(t.view(torch.uint8)).view(t.dtype).contiguous() if t.dtype == torch.float8_e4m3fn
                          else more(t).contiguous() for t in cache))
    want = as_values(cache)
    for s, n in enumerate(lens):
        for h in range(Hk):
            row = [(int(table[s][i // page]), i % page) for i in range(n)]
            keep = ref.kept_slots([cache.weight[p, h, r] for p, r in row], budget, recent)
            for j0 in range(0, len(keep), page):
                dp, part = int(dst[s][j0 // page]), [row[i] for i in keep[j0:j0 + page]]
                for name in ("k", "v"):
                    had = [float(cache.__getattribute__(name + "_scale")[p, h]) for p, _ in part]
                    top = max(had)
                    for i, (p, r) in enumerate(part):
                        want[name][dp, h, i] = ref.to_codes(getattr(cache, name)[p, h, r].double() * (had[i] / top))
                    want[name + "_scale"][dp, h] = top
                for i, (p, r) in enumerate(part):
                    want["pos"][dp, h, i] = int(cache.pos[p, h, r])
                    want["weight"][dp, h, i] = float(cache.weight[p, h, r])
    dev = to(cache, "cuda")
    new = kda.kda_cache_evict(dev, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), dst.cuda(), budget, recent)
    ok()
    assert new.tolist() == kept
    same_cache(dev, want)


@pytest.mark.parametrize("n,budget,recent", [(20_000, 150, 20), (300_000, 200, 7), (70_000, 60_000, 30_000)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_long_sequences(n, budget, recent, ties):
    """Several CTAs share a sequence, with more slots than they keep in shared memory."""
    page = 128
    cache, table = filled([n], 1, page, n)
    w = torch.rand(cache.weight.shape, generator=gen(3))
    w = torch.round(w * 40) if ties else w
    pages, need = cache.k.shape[0], -(-budget // page)
    dst = torch.arange(pages, pages + need, dtype=torch.int32)[None].contiguous()
    more = lambda t: torch.cat([t, torch.zeros((need, *t.shape[1:]), dtype=t.dtype)])  # noqa: E731
    dev = kda.KvCache(*(more(t.view(torch.uint8)).view(t.dtype) if t.dtype == torch.float8_e4m3fn else more(t)
                        for t in cache._replace(weight=w)))
    dev = to(dev, "cuda")
    kda.kda_cache_evict(dev, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), dst.cuda(), budget, recent)
    ok()
    flat = w[table[0, : -(-n // page)].long(), 0].reshape(-1)[:n]
    keep = torch.tensor(ref.kept_slots(flat.tolist(), budget, recent), dtype=torch.int32)
    assert torch.equal(dev.pos[pages:, 0].reshape(-1)[:budget].cpu(), keep)
    assert torch.equal(dev.weight[pages:, 0].reshape(-1)[:budget].cpu(), flat[keep.long()])


def test_evict_bad_pages_and_narrow_tables_are_reported():
    cache, table = filled([100], 1, 16, 1)
    lens = torch.tensor([100], dtype=torch.int32).cuda()
    base = cache.k.shape[0]
    pool = kda.KvCache(*(torch.cat([t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t] * 2) for t in cache))
    pool = pool._replace(k=pool.k.view(torch.float8_e4m3fn), v=pool.v.view(torch.float8_e4m3fn))
    good = torch.arange(base, base + 4, dtype=torch.int32)[None].contiguous()
    bad_src, bad_dst = table.clone(), good.clone()
    bad_src[0, 1], bad_dst[0, 2] = 12345, -1
    for src, dst in ((bad_src, good), (table, bad_dst), (table, good[:, :2].contiguous())):
        kda.kda_cache_evict(to(pool, "cuda"), src.cuda(), lens, dst.cuda(), 64, 8)
        assert kda.kda_device_status() == 1
    kda.kda_cache_evict(to(pool, "cuda"), table.cuda(), lens, good.cuda(), 64, 8)
    ok()


def test_evict_infinite_and_nan_weights():
    cache, table = filled([50], 1, 16, 1)
    w = torch.rand(cache.weight.shape, generator=gen(9))
    flat = [(int(table[0, i // 16]), i % 16) for i in range(50)]
    for i, x in ((3, float("nan")), (30, float("inf")), (31, -float("inf")), (8, float("inf"))):
        w[flat[i][0], 0, flat[i][1]] = x
    cache = cache._replace(weight=w)
    dst = torch.tensor([[cache.k.shape[0]]], dtype=torch.int32)
    one = lambda t: torch.cat([t, t[:1]]).contiguous()  # noqa: E731
    dev = kda.KvCache(*(one(t.view(torch.uint8)).view(t.dtype) if t.dtype == torch.float8_e4m3fn else one(t)
                        for t in cache))
    dev = to(dev, "cuda")
    kda.kda_cache_evict(dev, table.cuda(), torch.tensor([50], dtype=torch.int32).cuda(), dst.cuda(), 5, 2)
    ok()
    assert dev.pos[-1, 0, :5].tolist() == [3, 8, 30, 48, 49]


# ------------------------------------------------------------------ arguments

def test_tensors_are_checked_and_views_at_odd_places_taken():
    lens = [40, 9]
    cache, table = filled(lens, 2, 16, 30)
    q = randn(gen(8), 2, 4, D)
    want, tol, _, _ = ref.cached(cache, q, table, lens, SCALE, [1, 1])
    dev = to(cache, "cuda")
    # arrays that start 4 bytes into theirs, rows that start in the middle of theirs
    shift = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)  # noqa: E731
    qd = torch.cat([q, q, q]).cuda()[2:4]
    tab, n = shift(table.cuda()), shift(torch.tensor(lens, dtype=torch.int32).cuda())
    assert tab.data_ptr() % 16 == 4
    out = kda.kda_cache_attn(dev, qd, tab, n, SCALE)
    ok()
    within(out, want, tol, "out")
    good = dict(q=qd, block_table=tab, lens=n, scale=SCALE)
    for change, error in ((dict(q=qd.float()), TypeError), (dict(q=qd.transpose(0, 1)), ValueError),
                          (dict(q=torch.zeros((2, 8, D), dtype=torch.bfloat16, device="cuda")[:, ::2]), ValueError),
                          (dict(lens=n.long()), TypeError), (dict(lens=n[:1]), ValueError),
                          (dict(block_table=tab[0]), ValueError), (dict(lens=n.cpu()), ValueError),
                          (dict(out=torch.empty((2, 4, 64), dtype=torch.bfloat16, device="cuda")), ValueError),
                          (dict(slopes=torch.zeros(3, device="cuda")), ValueError), (dict(scale="x"), TypeError),
                          (dict(workspace=torch.empty(4, device="cuda")), TypeError)):
        with pytest.raises(error):
            kda.kda_cache_attn(dev, **{**good, **change})
    with pytest.raises(kda.KdaError) as e:
        kda.kda_cache_attn(dev, **good, cap=-1.0)
    assert e.value.status == 1
    with pytest.raises(kda.KdaError) as e:  # 3 heads over 2 KV heads
        kda.kda_cache_attn(dev, **{**good, "q": torch.zeros((2, 3, D), dtype=torch.bfloat16, device="cuda")})
    assert e.value.status == 1
    with pytest.raises(kda.KdaError) as e:
        kda.kda_attn_fwd(qd, qd, qd, SCALE, mask="prefix")
    assert e.value.status == 1
    with pytest.raises(ValueError, match="N is 3"):
        kda.kda_attn_fwd(qd, qd, qd, SCALE, N=3, cu_seqlens=cu_of([1, 1]).cuda())
    ok()


# ------------------------------------------------------------------ together

def test_the_layer_serves_a_prompt_and_its_continuation():
    """Prefill, append, decode with weights, evict, decode again: the example's path."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import attention_layer
    report = attention_layer.main(["--tokens", "300", "--steps", "6", "--budget", "128", "--recent", "32"])
    assert report["lens"] == [128 + report["after"]] * report["sequences"]
    assert report["finite"] and report["prefill_against_cache"] < 0.08
