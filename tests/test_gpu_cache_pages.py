"""Pages taken and given back on the device against lists on the host, and a serving loop that
uses all of the layers' operators together."""
import random

import pytest
import torch

import chunked_gated_delta_11_gb300 as kda
import recurrent_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    kda.build.build()
    kda.load()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def pool(seed, lens, page, width, spare):
    """Tables of the pages that the lengths need, the rest of a shuffled pool free."""
    r = random.Random(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    ids = list(range(pages))
    r.shuffle(ids)
    table = []
    for n in need:
        table.append([ids.pop() for _ in range(n)] + [-1] * (width - n))
    count = len(ids)
    return table, ids + [-7] * (pages - count), count, pages


def check_reserve(table, lens, new, free, count, page, pages, rows=None, **kw):
    rows = sum(new) if rows is None else rows
    t, left = ints(table), ints([count])
    r = kda.kda_cache_reserve(t, ints(lens), ints(new), ints(free), left, page, rows=rows, **kw)
    assert kda.kda_device_status() == 0
    want = ref.reserve(table, lens, new, free, count, page, rows, pages)
    got = (t.tolist(), r.lens.tolist(), r.cu_seqlens.tolist(), r.slots.tolist(), r.free_count.item())
    for name, g, w in zip(("table", "lens", "cu_seqlens", "slots", "free_count"), got, want):
        assert g == w, name
    return got


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("seed", range(6))
def test_reserve(page, seed):
    r = random.Random(100 * page + seed)
    N = r.choice([1, 3, 40])
    lens = [r.choice([0, 1, page - 1, page, page + 1, r.randrange(300)]) for _ in range(N)]
    new = [r.choice([0, 0, 1, page, page + 3, r.randrange(500)]) for _ in range(N)]
    width = max(1, max(-(-(a + b) // page) for a, b in zip(lens, new)) - r.choice([0, 0, 2]))
    width = max(width, max(-(-a // page) for a in lens))
    need = sum(-(-(a + b) // page) + (a // -page) for a, b in zip(lens, new))
    table, free, count, pages = pool(seed, lens, page, width, max(0, need - r.choice([0, 0, 1, need // 2])))
    check_reserve(table, lens, new, free, count, page, pages, rows=sum(new) + r.choice([0, 0, 5]))


def test_reserve_many_sequences_and_rows():
    r = random.Random(1)
    for N, most in ((3000, 3), (1100, 0), (70, 900), (16384, 1)):
        lens = [r.randrange(40) for _ in range(N)]
        new = [r.randint(0, most) for _ in range(N)]
        page = 16
        width = max(-(-(a + b) // page) for a, b in zip(lens, new))
        need = sum(-(-(a + b) // page) + (a // -page) for a, b in zip(lens, new))
        table, free, count, pages = pool(N, lens, page, width, need - need // 5)
        check_reserve(table, lens, new, free, count, page, pages)


@pytest.mark.parametrize("N,most", [(5, 40), (300, 60)])
def test_reserve_in_place(N, most):
    r = random.Random(N)
    lens, new = [r.randrange(50) for _ in range(N)], [r.randrange(most) for _ in range(N)]
    table, free, count, pages = pool(2, lens, 32, 8, N)
    want = ref.reserve(table, lens, new, free, count, 32, sum(new), pages)
    t, held, left = ints(table), ints(lens), ints([count])
    got = kda.kda_cache_reserve(t, held, ints(new), ints(free), left, 32, rows=sum(new), new_lens=held, new_free_count=left)
    assert kda.kda_device_status() == 0
    assert got.lens.data_ptr() == held.data_ptr() and got.free_count.data_ptr() == left.data_ptr()
    assert (t.tolist(), held.tolist(), got.slots.tolist(), left.item()) == (want[0], want[1], want[3], want[4])


def test_reserve_without_slots():
    lens, new = [5, 0, 40], [100, 3, 0]
    table, free, count, pages = pool(3, lens, 16, 8, 20)
    want = ref.reserve(table, lens, new, free, count, 16, 103, pages)
    t = ints(table)
    r = kda.kda_cache_reserve(t, ints(lens), ints(new), ints(free), ints([count]), 16)
    assert kda.kda_device_status() == 0
    assert r.slots is None and (t.tolist(), r.lens.tolist(), r.free_count.item()) == (want[0], want[1], want[4])


@pytest.mark.parametrize("what", ["length", "negative length", "negative rows", "rows", "count", "negative count", "page", "free page"])
def test_reserve_bad_values_are_latched(what):
    lens, new, width, page = [20, 30, 5], [10, 20, 40], 6, 16
    table, free, count, pages = pool(4, lens, page, width, 9)
    rows = sum(new)
    if what == "length":
        lens[1] = width * page + 1
    elif what == "negative length":
        lens[1] = -3
    elif what == "negative rows":
        new[1] = -20
    elif what == "rows":
        rows -= 15
    elif what == "count":
        count = pages + 1
    elif what == "negative count":
        count = -1
    elif what == "page":
        table[1][1] = pages
    else:
        free[count - 1] = -1
    big = torch.full((rows + 8,), 99, dtype=torch.int64, device="cuda")
    edge = ints(table + [[55] * width])
    r = kda.kda_cache_reserve(edge[:3], ints(lens), ints(new), ints(free), ints([count]), page, rows=rows, slots=big[:rows])
    assert kda.kda_device_status() == 1
    assert (big[rows:] == 99).all() and (edge[3] == 55).all()
    cu, slots = r.cu_seqlens.tolist(), r.slots.tolist()
    assert cu[0] == 0 and all(a <= b for a, b in zip(cu, cu[1:])) and cu[-1] <= rows
    assert all(-1 <= s < pages * page for s in slots)
    assert 0 <= r.free_count.item() <= pages
    if what in ("length", "negative length"):
        assert slots[10:30] == [-1] * 20 and r.lens.tolist()[1] == lens[1]


@pytest.mark.parametrize("seed", range(8))
def test_release(seed):
    r = random.Random(seed)
    page = r.choice([16, 64])
    N = r.choice([1, 5, 60, 2000])
    lens = [r.choice([0, 1, page, page + 1, r.randrange(400)]) for _ in range(N)]
    keep = [r.choice([0, n, max(0, n - 1), max(0, n - page), n + 5, r.randrange(n + 1)]) for n in lens] if seed % 2 else None
    width = max(1, max(-(-n // page) for n in lens)) + r.choice([0, 2])
    table, free, count, pages = pool(seed, lens, page, width, 6)
    left, listed = ints([count]), ints(free)
    out = kda.kda_cache_release(ints(table), ints(lens), listed, left, page, keep=None if keep is None else ints(keep),
                                **(dict(new_free_count=left) if seed % 3 == 0 else {}))
    assert kda.kda_device_status() == 0
    want = ref.release(table, lens, free, count, page, keep)
    assert (listed.tolist(), out.item()) == want
    assert (out.data_ptr() == left.data_ptr()) == (seed % 3 == 0)


@pytest.mark.parametrize("what", ["length", "page", "no room", "count"])
def test_release_bad_values_are_latched(what):
    lens, page, width = [40, 20], 16, 4
    table, free, count, pages = pool(5, lens, page, width, 2)
    if what == "length":
        lens[0] = width * page + 9
    elif what == "page":
        table[0][1] = -9
    elif what == "no room":
        count += 3
    else:
        count = -2
    listed = torch.cat([ints(free), ints([77, 77])])
    out = kda.kda_cache_release(ints(table), ints(lens), listed[:pages], ints([count]), page)
    assert kda.kda_device_status() == 1
    assert (listed[pages:] == 77).all() and 0 <= out.item() <= pages
    if what == "page":
        assert -1 in listed[:pages].tolist() and -9 not in listed.tolist()


def test_taken_and_given_back_again_and_again():
    r = random.Random(9)
    N, page, width, pages = 12, 16, 20, 150
    free, count = ints(r.sample(range(pages), pages)), ints([pages])
    table, lens = ints([[-1] * width] * N), ints([0] * N)
    for _ in range(30):
        new = [r.choice([0, 1, 20, 90]) for _ in range(N)]
        got = kda.kda_cache_reserve(table, lens, ints(new), free, count, page, rows=sum(new), new_lens=lens, new_free_count=count)
        held = [t[: -(-n // page)] for t, n in zip(table.tolist(), lens.tolist())]
        used = [p for t in held for p in t]
        assert sorted(used + free.tolist()[: count.item()]) == list(range(pages))
        assert len([s for s in got.slots.tolist() if s >= 0]) == len({s for s in got.slots.tolist() if s >= 0})
        keep = [r.choice([n, n, n // 2, 0]) for n in lens.tolist()]
        kda.kda_cache_release(table, lens, free, count, page, keep=ints(keep), new_free_count=count)
        lens = ints(keep)
    assert kda.kda_device_status() == 0


def test_refusals():
    table, lens, free, count = ints([[0, 1]]), ints([5]), ints([2, 3]), ints([2])
    with pytest.raises(ValueError, match="slots needs rows"):
        kda.kda_cache_reserve(table, lens, ints([1]), free, count, 16, slots=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        kda.kda_cache_reserve(table, lens, ints([1, 2]), free, count, 16, rows=3)
    with pytest.raises(TypeError, match="int32"):
        kda.kda_cache_reserve(table, lens.long(), ints([1]), free, count, 16, rows=1)
    with pytest.raises(ValueError, match="out of range"):
        kda.kda_cache_reserve(table, lens, ints([1]), free, count, 16, rows=-1)
    with pytest.raises(kda.KdaError, match="UNSUPPORTED"):
        kda.kda_cache_reserve(table, lens, ints([1]), free, count, 20, rows=1)
    with pytest.raises(kda.KdaError, match="INVALID_ARG"):
        kda.kda_cache_release(table, lens, free, count, 16, new_free_count=free[:1])
    assert kda.kda_device_status() == 0


def test_a_serving_loop():
    """Prompts and tokens of a hybrid model's layers: convolution, KDA, state-space layer, and attention
    over a cache whose pages are taken and given back on the device, against one pass over all."""
    N, H, Hk, D, P, S, page, width, scale = 3, 2, 1, 128, 64, 64, 16, 8, 128 ** -0.5
    lens = [70, 3, 41]
    steps, T = 5, sum(lens)
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    C = 3 * H * D
    w = randn(C, 4)
    A, skip = -torch.rand(H, generator=g, device="cuda"), torch.rand(H, generator=g, device="cuda")
    total = [n + steps for n in lens]
    # every sequence's rows in full, and the calls that see them in parts
    full = {k: [randn(n, *s) for n in total] for k, s in dict(rows=(C,), gate=(H, D), beta=(H,), x=(H, P), dt=(H,), B=(1, S),
                                                              C=(1, S), k=(Hk, D), v=(Hk, D)).items()}

    def part(a, b):  # tokens [a_n, b_n) of every sequence, packed
        return {k: torch.cat([t[i:j] for t, i, j in zip(v, a, b)]).contiguous() for k, v in full.items()}

    def recurrent(p, cu, conv, s, m, decode):
        rows, conv = kda.kda_conv_fwd(p["rows"], w, initial_state=conv, cu_seqlens=cu)
        q, k, v = (t.contiguous() for t in rows.view(-1, 3, H, D).unbind(1))
        run = kda.kda_decode if decode else kda.kda_fwd_fused
        o, s = run(q, k, v, p["gate"], p["beta"], scale, -5.0, initial_state=s, cu_seqlens=cu)
        ssm = kda.kda_ssm_step if decode else kda.kda_ssm_fwd
        y, m = ssm(p["x"], p["dt"], A, p["B"], p["C"], skip, initial_state=m, cu_seqlens=cu)
        return q, o, y, conv, s, m

    cu_all = ints([0, *torch.tensor(total).cumsum(0).tolist()])
    q, o, y, conv_w, s_w, m_w = recurrent(part([0] * N, total), cu_all, None, None, None, False)
    attn_w = kda.kda_attn_fwd(q, part([0] * N, total)["k"], part([0] * N, total)["v"], scale, cu_seqlens=cu_all)

    cache = kda.kda_cache_alloc(40, Hk, page)
    free, count = torch.randperm(40, generator=g, device="cuda").int(), ints([40])
    table, held = ints([[-1] * width] * N), ints([0] * N)
    state, a = (None, None, None), [0] * N
    for step in range(steps + 1):
        b = lens if step == 0 else [n + 1 for n in a]
        p, new = part(a, b), [j - i for i, j in zip(a, b)]
        r = kda.kda_cache_reserve(table, held, ints(new), free, count, page, rows=sum(new), new_free_count=count)
        assert r.cu_seqlens.tolist() == [0, *torch.tensor(new).cumsum(0).tolist()]
        q1, o1, y1, *state = recurrent(p, r.cu_seqlens, *state, decode=step > 0)
        kda.kda_cache_append(cache, p["k"], p["v"], table, held, cu_seqlens=r.cu_seqlens)
        held = r.lens
        at = kda.kda_cache_attn(cache, q1, table, held, scale, cu_seqlens=r.cu_seqlens, accumulate=True)
        # the slots are where the rows went
        page_of, place = r.slots // page, r.slots % page
        codes = cache.v[page_of, 0, place].float() * cache.v_scale[page_of, 0][:, None]
        assert ((codes - p["v"][:, 0].float()).norm() / codes.norm()) < 0.06
        rows = torch.cat([torch.arange(c + i, c + j) for c, i, j in zip(cu_all.tolist(), a, b)]).cuda()
        for got, want, tol in ((o1, o, 1e-2), (y1, y, 1e-2), (at, attn_w, 8e-2)):
            assert ((got.float() - want[rows].float()).norm() / want[rows].float().norm()) < tol
        a = b
    for got, want, tol in zip(state, (conv_w, s_w, m_w), (0.0, 1e-2, 1e-4)):
        assert ((got.float() - want.float()).norm() / want.float().norm()) <= tol
    # eviction into pages of its own, and the old ones back
    budget = 32
    dst = ints([[-1] * 2] * N)
    fits = kda.kda_cache_reserve(dst, ints([0] * N), held.clamp(max=budget), free, count, page, new_free_count=count)
    kept = kda.kda_cache_evict(cache, table, held, dst, budget, 8)
    kda.kda_cache_release(table, held, free, count, page, new_free_count=count)
    assert torch.equal(kept, fits.lens) and kda.kda_device_status() == 0
    used = [t for row, n in zip(dst.tolist(), kept.tolist()) for t in row[: -(-n // page)]]
    assert sorted(used + free.tolist()[: count.item()]) == list(range(40))
