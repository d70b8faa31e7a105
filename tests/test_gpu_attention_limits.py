"""The attention operators at the limits of what their contracts allow: caps of any size, keys that a row does not
see, scales far apart, lengths in place, caches that were evicted from."""
import itertools
import math

import pytest
import torch

import attn_ref as ref
import chunked_gated_delta_11_gb300 as kda

pytestmark = pytest.mark.gpu

D = 128
SCALE = D ** -0.5
SCALE32 = float(torch.tensor(SCALE, dtype=torch.float32))


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


def ints(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def ok():
    assert kda.kda_device_status() == 0


def within(got, want, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    over = ((got - want).abs() - tol).max().item()
    assert over <= 0, f"{what}: {over:.3e} over the tolerance"


def to(cache, device):
    return kda.KvCache(*(t.to(device) for t in cache))


# ------------------------------------------------------------------ caps of any size
# A capped score is off by its fp32 roundings, which are relative to |q||k| and to the score; a cap of at most 128
# adds up to 2.2e-6 of itself (the fitted tanh of the prefill).  No term grows with a larger cap.

CAPS = [1e-39, 1e-20, 0.5, 50.0, 128.0, 129.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e30, 3e38]


def capped(x, cap):
    c = float(torch.tensor(cap, dtype=torch.float32))
    return c * torch.tanh(x / c)


def cap_error(cap):
    return 2.2e-6 * min(cap, 128.0)


@pytest.mark.parametrize("cap", CAPS)
def test_prefill_cap(cap):
    n, g = 400, gen(1)
    q, k, v = 4 * randn(g, n, 1, D), randn(g, n, 1, D), randn(g, n, 1, D)
    out = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), SCALE, cap=cap)
    ok()
    qd, kd, vd = (t[:, 0].double() for t in (q, k, v))
    x = SCALE32 * (qd @ kd.T)
    d = 160 * ref.F32 * (SCALE32 * (qd.abs() @ kd.abs().T) + x.abs()) + cap_error(cap)
    seen = torch.ones(n, n, dtype=torch.bool).tril()
    p = capped(x, cap).masked_fill(~seen, -torch.inf).softmax(1)
    d = 4 * d.masked_fill(~seen, 0.0).amax(1, keepdim=True)
    want = p @ vd
    tol = ref.BF16 * want.abs() * (1 + ref.BF16) + (ref.BF16 + d + 2.0 ** -15) * (p @ vd.abs())
    within(out[:, 0], want, tol, "out")


@pytest.mark.parametrize("H", [1, 12, 24])
@pytest.mark.parametrize("cap", CAPS)
def test_cached_cap(cap, H):
    n, g = 300, gen(2)
    q = 4 * randn(g, 1, H, D)
    cache = kda.kda_cache_alloc(5, 1, 64, device="cpu")
    for t in (cache.k, cache.v):
        t.copy_(torch.randn(t.shape, generator=g).to(torch.float8_e4m3fn))
    table = torch.arange(5, dtype=torch.int32)[None]
    dev = to(cache, "cuda")
    out = kda.kda_cache_attn(dev, q.cuda(), table.cuda(), ints(n), SCALE, cap=cap, accumulate=True)
    ok()
    k, v = (t.double().view(-1, D)[:n] for t in (cache.k, cache.v))
    x = SCALE32 * (q[0].double() @ k.T)
    d = 160 * ref.F32 * (SCALE32 * (q[0].double().abs() @ k.abs().T) + x.abs()) + cap_error(cap)
    p = capped(x, cap).softmax(1)
    d = 4 * d.amax(1, keepdim=True)
    want = p @ v
    tol = ref.BF16 * want.abs() * (1 + ref.BF16) + (ref.F16 + d + 2.0 ** -15) * (p @ v.abs()) \
        + 4 * 2.0 ** -25 * p.amax(1, keepdim=True) * v.abs().sum(0)
    within(out[0], want, tol, "out")
    total = p.sum(0)
    addtol = ((d + 8 * ref.F32) * p).sum(0) + (H + 4) * ref.F32 * total
    within(dev.weight.view(-1)[:n], total, addtol, "weight")


def one_key(cap, part, n):
    """A key of capped score L at distance n - 1 against the query's own key of score 0, which a bias brings to 3
    below it: its weight shows the error of L.  Query's and key's channel 0, the slope, the weight, its score error."""
    b = 256.0
    a = float(torch.tensor(part * cap / (SCALE32 * b), dtype=torch.bfloat16))
    x = torch.tensor(SCALE32 * a * b, dtype=torch.float64)
    score = float(capped(x, cap))
    slope = float(torch.tensor((score + 3.0) / (n - 1), dtype=torch.float32))
    # the keys between have scores of 0 and their own distances
    gap = torch.arange(n, dtype=torch.float64)
    s = -slope * gap
    s[n - 1] += score
    return a, b, slope, s.softmax(0)[n - 1], 24 * ref.F32 * (abs(float(x)) + abs(score)) + cap_error(cap)


@pytest.mark.parametrize("cap", [100.0, 1000.0, 4000.0, 8000.0, 1e5])
@pytest.mark.parametrize("part", [0.03, 0.1, 0.2, 0.3, 0.36, 0.5, 0.65, 0.9])
@pytest.mark.parametrize("n", [2, 300])
def test_prefill_large_scores_under_a_cap(cap, part, n):
    a, b, slope, weight, d = one_key(cap, part, n)
    q, k, v = (torch.zeros(n, 1, D, dtype=torch.bfloat16) for _ in range(3))
    q[:, 0, 0], k[0, 0, 0], v[0] = a, b, 1.0
    out = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), SCALE, cap=cap, slopes=torch.tensor([slope]).cuda())
    ok()
    within(out[-1, 0], weight.expand(D), (2.02 * ref.BF16 + 2 * d) * weight, "out")


@pytest.mark.parametrize("cap", [100.0, 1000.0, 4000.0, 8000.0, 1e5])
@pytest.mark.parametrize("part", [0.03, 0.1, 0.2, 0.3, 0.36, 0.5, 0.65, 0.9])
def test_cached_large_scores_under_a_cap(cap, part):
    n = 300
    a, b, slope, weight, d = one_key(cap, part, n)
    cache = kda.kda_cache_alloc(5, 1, 64, device="cpu")
    cache.k.view(-1, D)[0, 0] = b
    cache.pos.view(-1)[:n] = torch.arange(n, dtype=torch.int32)
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16)
    q[0, 0, 0] = a
    dev = to(cache, "cuda")
    kda.kda_cache_attn(dev, q.cuda(), torch.arange(5, dtype=torch.int32)[None].cuda(), ints(n), SCALE, cap=cap,
                       slopes=torch.tensor([slope]).cuda(), accumulate=True)
    ok()
    within(dev.weight.view(-1)[:1], weight[None], (2 * d + 64 * ref.F32) * weight, "weight")


@pytest.mark.parametrize("cap", [1e-39, 1e-37, 1e-20])
def test_zero_scores_under_a_tiny_cap(cap):
    n, g = 200, gen(16)
    zero, v = torch.zeros(n, 1, D, dtype=torch.bfloat16), randn(g, n, 1, D)
    out = kda.kda_attn_fwd(zero.cuda(), randn(g, n, 1, D).cuda(), v.cuda(), SCALE, mask="full", cap=cap)
    ok()
    mean, size = v[:, 0].double().mean(0), v[:, 0].double().abs().mean(0)
    within(out[:, 0], mean.expand(n, D), ref.BF16 * mean.abs() * (1 + ref.BF16) + (ref.BF16 + 2.0 ** -15) * size, "prefill")
    cache = kda.kda_cache_alloc(4, 1, 64)
    table = torch.arange(4, dtype=torch.int32)[None].cuda()
    kda.kda_cache_append(cache, v.cuda(), v.cuda(), table, ints(0))
    kda.kda_cache_attn(cache, zero[:1].cuda(), table, ints(n), SCALE, cap=cap, accumulate=True)
    ok()
    within(cache.weight.view(-1)[:n], torch.full((n,), 1.0 / n, dtype=torch.float64), 64 * ref.F32 / n, "weight")


# ------------------------------------------------------------------ scales far apart

@pytest.mark.parametrize("H", [1, 12, 24])
@pytest.mark.parametrize("small,large", [(None, 70), (None, 110), (-60, 40), (-50, 110), (-60, 30)])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
def test_cached_blocks_of_scales_far_apart(H, small, large, order):
    """Blocks of tiny (None: zero) values beside blocks of huge ones: all count in the denominator."""
    n, page, g = 640, 16, gen(11)
    blocks = n // page
    huge = {"up": [j >= blocks // 2 for j in range(blocks)], "down": [j < blocks // 2 for j in range(blocks)],
            "mixed": [j % 3 == 1 for j in range(blocks)]}[order]
    k, v = randn(g, n, 1, D), torch.randn((n, 1, D), generator=g)
    for j, h in enumerate(huge):
        v[j * page:(j + 1) * page] *= 2.0 ** large if h else 0.0 if small is None else 2.0 ** small
    cache = kda.kda_cache_alloc(blocks, 1, page)
    table = torch.arange(blocks, dtype=torch.int32)[None]
    kda.kda_cache_append(cache, k.cuda(), v.to(torch.bfloat16).cuda(), table.cuda(), ints(0))
    q = randn(g, 1, H, D)
    here = to(cache, "cpu")
    want, tol, add, addtol = ref.cached(here, q, table, [n], SCALE, [1])
    out = kda.kda_cache_attn(cache, q.cuda(), table.cuda(), ints(n), SCALE, accumulate=True)
    ok()
    within(out, want, tol, "out")
    within(cache.weight, add, addtol + 4 * ref.F32 * add, "weight")


@pytest.mark.parametrize("scale", [0.0, 1e-40])
def test_cached_blocks_without_a_normal_scale_are_left_out(scale):
    n, page, g = 96, 16, gen(12)
    cache = kda.kda_cache_alloc(6, 1, page)
    table = torch.arange(6, dtype=torch.int32)[None]
    kda.kda_cache_append(cache, randn(g, n, 1, D).cuda(), randn(g, n, 1, D).cuda(), table.cuda(), ints(0))
    cache.v_scale[2] = scale
    q = randn(g, 1, 4, D)
    left = to(cache, "cpu")
    left.pos[2] = n  # after the query
    want, tol, add, addtol = ref.cached(left, q, table, [n], SCALE, [1])
    out = kda.kda_cache_attn(cache, q.cuda(), table.cuda(), ints(n), SCALE, accumulate=True)
    ok()
    within(out, want, tol, "out")
    within(cache.weight, add, addtol + 4 * ref.F32 * add, "weight")


# ------------------------------------------------------------------ lengths

@pytest.mark.parametrize("count", [1, 3, 40])
def test_append_to_a_negative_length_writes_nothing(count):
    g = gen(8)
    rows = [0, count, 2 * count]
    cache = kda.kda_cache_alloc(12, 2, 16)
    table = torch.arange(12, dtype=torch.int32).view(2, 6).cuda()
    kda.kda_cache_append(cache, *(randn(g, 40, 2, D).cuda() for _ in range(2)), table, ints(0, 0), positions=ints(*range(40)))
    was = [t.clone() for t in cache]
    k, v = (randn(g, 2 * count, 2, D).cuda() for _ in range(2))
    kda.kda_cache_append(cache, k, v, table, ints(-4, 20), cu_seqlens=ints(*rows))
    assert kda.kda_device_status() == 1
    for now, old in zip(cache, was):
        assert torch.equal(now.view(torch.uint8)[:6], old.view(torch.uint8)[:6])
    assert not torch.equal(cache.pos[6:], was[4][6:])


@pytest.mark.parametrize("lens,budget,recent", [([40_000], 300, 20), ([900, 10, 5000, 300] * 8, 256, 64)])
def test_evict_lengths_in_place(lens, budget, recent):
    """new_lens may be the tensor of the lengths."""
    page, Hk = 64, 4
    need = [-(-n // page) for n in lens]
    keep = [-(-min(n, budget) // page) for n in lens]
    pages = sum(need) + sum(keep)
    ids = torch.arange(pages, dtype=torch.int32)

    def table_of(counts, first):
        t = torch.full((len(counts), max(counts)), -1, dtype=torch.int32)
        for row, m in zip(t, counts):
            row[:m] = ids[first:first + m]
            first += m
        return t.cuda()

    src, dst = table_of(need, 0), table_of(keep, sum(need))
    made = kda.kda_cache_alloc(pages, Hk, page)
    made.k.view(torch.uint8).copy_(torch.randint(0, 120, made.k.shape, generator=gen(9), dtype=torch.uint8))
    made.pos.copy_(torch.arange(made.pos.numel(), dtype=torch.int32).view(made.pos.shape))
    made.weight.copy_(torch.rand(made.weight.shape, generator=gen(10)))
    want, got = kda.KvCache(*(t.clone() for t in made)), kda.KvCache(*(t.clone() for t in made))
    new = kda.kda_cache_evict(want, src, ints(*lens), dst, budget, recent)
    mine = ints(*lens)
    assert kda.kda_cache_evict(got, src, mine, dst, budget, recent, new_lens=mine) is not None
    ok()
    assert torch.equal(mine, new) and new.tolist() == [min(n, budget) for n in lens]
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ positions

def test_cached_single_tokens_see_no_later_position():
    """The newest slot's position is the query's, whatever the other slots hold; the ways to say so agree."""
    g, n = gen(13), [200, 77]
    cache = kda.kda_cache_alloc(8, 2, 64)
    table = torch.arange(8, dtype=torch.int32).view(2, 4)
    order = torch.cat([torch.randperm(m, generator=g) for m in n]).to(torch.int32)
    kda.kda_cache_append(cache, randn(g, sum(n), 2, D).cuda(), randn(g, sum(n), 2, D).cuda(), table.cuda(), ints(0, 0),
                         positions=order.cuda(), cu_seqlens=cu_of(n).cuda())
    q = randn(g, 2, 8, D)
    want, tol, add, addtol = ref.cached(to(cache, "cpu"), q, table, n, SCALE, [1, 1])
    assert (add == 0).sum() > (n[0] + n[1]) // 4
    call = lambda **kw: kda.kda_cache_attn(cache, q.cuda(), table.cuda(), ints(*n), SCALE, **kw)  # noqa: E731
    plain = call(accumulate=True)
    within(plain, want, tol, "out")
    within(cache.weight, add, addtol + 4 * ref.F32 * add, "weight")
    for kw in (dict(cu_seqlens=ints(0, 1, 2)), dict(positions=ints(int(order[199]), int(order[276]))),
               dict(slopes=torch.zeros(8).cuda())):
        assert torch.equal(call(**kw), plain)
    ok()


@pytest.mark.parametrize("counts", [[1, 1], [1, 4]])
def test_a_cache_that_was_evicted_from(counts):
    """After eviction every KV head has slots and positions of its own; new tokens are appended and attended to."""
    n, page, Hk, H, budget = [500, 333], 64, 2, 8, 130
    g = gen(14)
    cache = kda.kda_cache_alloc(32, Hk, page)
    table = torch.arange(32, dtype=torch.int32).view(2, 16)
    src, dst = table[:, :8].contiguous(), table[:, 8:].contiguous()
    rows = lambda m: [randn(g, m, Hk, D).cuda() for _ in range(2)]  # noqa: E731
    kda.kda_cache_append(cache, *rows(sum(n)), src.cuda(), ints(0, 0), cu_seqlens=cu_of(n).cuda())
    kda.kda_cache_attn(cache, 4 * randn(g, 2, H, D).cuda(), src.cuda(), ints(*n), SCALE, accumulate=True)
    lens = kda.kda_cache_evict(cache, src.cuda(), ints(*n), dst.cuda(), budget, 20)
    positions = [n[s] + i for s, c in enumerate(counts) for i in range(c)]
    kda.kda_cache_append(cache, *rows(sum(counts)), dst.cuda(), lens, positions=ints(*positions),
                         cu_seqlens=cu_of(counts).cuda())
    ok()
    lens = [m + c for m, c in zip(lens.tolist(), counts)]
    here = to(cache, "cpu")
    assert lens == [budget + c for c in counts]
    assert not torch.equal(here.pos[8, 0], here.pos[8, 1])
    q = 2 * randn(g, sum(counts), H, D)
    slopes = 0.05 * torch.rand(H, generator=g)
    for bias in (None, slopes):
        for at in (None, torch.tensor(positions, dtype=torch.int32)):
            was = cache.weight.double().cpu()
            want, tol, add, addtol = ref.cached(here, q, dst, lens, SCALE, counts, slopes=bias, positions=at)
            out = kda.kda_cache_attn(cache, q.cuda(), dst.cuda(), ints(*lens), SCALE, accumulate=True,
                                     slopes=None if bias is None else bias.cuda(),
                                     positions=None if at is None else at.cuda(), cu_seqlens=cu_of(counts).cuda())
            ok()
            within(out, want, tol, "out")
            within(cache.weight, was + add, addtol + 4 * ref.F32 * (was + add), "weight")


# ------------------------------------------------------------------ what a row does not see

def prefill_inputs(seed, T, H, Hk):
    g = gen(seed)
    return [x.cuda() for x in (3 * randn(g, T, H, D), randn(g, T, Hk, D), randn(g, T, Hk, D))]


# one CTA to a piece of work, several pieces to a CTA, several CTAs to a piece
SHAPES = [([130, 70, 300], 2, 1), ([90, 257, 31, 500] * 12, 8, 2), ([1500, 1000], 1, 1)]


@pytest.mark.parametrize("lengths,H,Hk", SHAPES, ids=["one", "more", "share"])
@pytest.mark.parametrize("mask", ["causal", "full", "prefix"])
@pytest.mark.parametrize("cap,slope", [(0.0, None), (20.0, None), (0.0, 0.1), (1000.0, 0.1)])
def test_prefill_other_sequences_change_no_bit(lengths, H, Hk, mask, cap, slope):
    q, k, v = prefill_inputs(3, sum(lengths), H, Hk)
    cu = cu_of(lengths)
    slopes = None if slope is None else torch.full((H,), slope).cuda()
    prefix = ints(*[n // 3 for n in lengths]) if mask == "prefix" else None
    call = lambda: kda.kda_attn_fwd(q, k, v, SCALE, mask=mask, cap=cap, slopes=slopes, prefix_lens=prefix,  # noqa: E731
                                    cu_seqlens=cu.cuda())
    want = call()
    odd = torch.zeros(sum(lengths), dtype=torch.bool)
    for s in range(1, len(lengths), 2):
        odd[cu[s]:cu[s + 1]] = True
    odd = odd.cuda()
    kept = [x.clone() for x in (q, k, v)]
    for size in (0.0, 1.0, 50.0):
        for mine in (odd, ~odd):
            for x, old, new in zip((q, k, v), kept, prefill_inputs(4, sum(lengths), H, Hk)):
                x.copy_(torch.where(mine[:, None, None], new * size, old))
            got = call()
            assert torch.equal(got[~mine], want[~mine]), size
    ok()


@pytest.mark.parametrize("lengths,H,Hk", [([700], 2, 1), ([700, 500] * 15, 8, 2), ([2100], 1, 1)],
                         ids=["one", "more", "share"])
@pytest.mark.parametrize("cap,slope", [(0.0, None), (20.0, None), (0.0, 0.1), (1000.0, 0.1)])
def test_prefill_later_tokens_change_no_bit(lengths, H, Hk, cap, slope):
    q, k, v = prefill_inputs(5, sum(lengths), H, Hk)
    cu = cu_of(lengths).cuda()
    slopes = None if slope is None else torch.full((H,), slope).cuda()
    call = lambda: kda.kda_attn_fwd(q, k, v, SCALE, cap=cap, slopes=slopes, cu_seqlens=cu)  # noqa: E731
    want = call()
    kept = [x.clone() for x in (q, k, v)]
    last = sum(lengths) - lengths[-1]
    for size in (0.0, 1.0, 50.0):
        for at in (1, 37, 128, 300, 450):
            for x, old, new in zip((q, k, v), kept, prefill_inputs(6, sum(lengths), H, Hk)):
                x.copy_(old)
                x[last + at:] = new[last + at:] * size
            assert torch.equal(call()[:last + at], want[:last + at]), (size, at)
    ok()


@pytest.mark.parametrize("where", [slice(0, 700), slice(700, 1400), slice(1400, 2100), slice(0, 2100), slice(1000, 1001)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("which", ["k", "v"])
def test_prefill_nan_keys_and_values_show(where, cap, which):
    """A visible NaN key or value makes a row NaN, whether one CTA or several take its piece of work."""
    n = 2100
    for H in (1, 64):
        q, k, v = prefill_inputs(7, n, H, 1)
        (k if which == "k" else v)[where] = float("nan")
        out = kda.kda_attn_fwd(q, k, v, SCALE, mask="full", cap=cap)
        ok()
        assert torch.isnan(out).all(), H


# ------------------------------------------------------------------ arguments

def small_cache():
    g = gen(15)
    cache = kda.kda_cache_alloc(4, 1, 16)
    table = torch.arange(4, dtype=torch.int32)[None].cuda()
    kda.kda_cache_append(cache, randn(g, 40, 1, D).cuda(), randn(g, 40, 1, D).cuda(), table, ints(0))
    return cache, table, randn(g, 1, 4, D).cuda()


def test_accumulate_that_is_no_truth_value_is_refused():
    cache, table, q = small_cache()
    with pytest.raises(TypeError, match="accumulate"):
        kda.kda_cache_attn(cache, q, table, ints(40), SCALE, accumulate=torch.zeros(2))
    ok()


@pytest.mark.parametrize("recent", [0, 5, 2 ** 31 - 1])
def test_evict_a_budget_beyond_the_table_copies_everything(recent):
    cache, table, _ = small_cache()
    cache.weight.copy_(torch.rand(cache.weight.shape))
    many = kda.KvCache(*(torch.cat([t.view(torch.uint8)] * 2).view(t.dtype) for t in cache))
    src = torch.full((64, 4), -1, dtype=torch.int32, device="cuda")
    src[5] = table[0]
    lens = torch.zeros(64, dtype=torch.int32, device="cuda")
    lens[5] = 40
    new = kda.kda_cache_evict(many, src, lens, torch.where(src >= 0, src + 4, -1), 2 ** 31 - 1, recent)
    ok()
    assert torch.equal(new, lens)
    for t in many:
        x = t.view(torch.uint8).reshape(8, 16, -1) if t.dim() > 2 else t
        assert torch.equal(x[4:6], x[:2]) and torch.equal(x[6, :8] if t.dim() > 2 else x[6], x[2, :8] if t.dim() > 2 else x[2])


def test_running_out_of_memory_is_torchs_error():
    cache, _, q = small_cache()
    wide = torch.full((1, 1 << 26), -1, dtype=torch.int32, device="cuda")  # 2^30 slots: 550 GB for the splits of 64 heads
    q = q.repeat(1, 1, 1).expand(256, 4, D).contiguous()
    with pytest.raises(torch.OutOfMemoryError):
        kda.kda_cache_attn(cache, q, wide, ints(40), SCALE, accumulate=True)
    ok()
