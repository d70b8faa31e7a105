"""Pages that are not there: ids outside the pool, and pools that run out in the middle of a batch."""
import pytest
import torch

import chunked_gated_delta_11_gb300 as kda
from test_gpu_cache_pages import check_reserve, ints, pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    kda.build.build()
    kda.load()


@pytest.mark.parametrize("bad", [-9, 1 << 30])
def test_an_id_outside_the_pool_does_not_reach_the_table(bad):
    lens, new, width, page = [20, 30, 5], [10, 20, 40], 6, 16
    table, free, count, pages = pool(4, lens, page, width, 9)
    assert bad < 0 or bad >= pages
    free[count - 2] = bad   # the second page that is taken: sequence 1's
    t = ints(table)
    r = kda.kda_cache_reserve(t, ints(lens), ints(new), ints(free), ints([count]), page, rows=sum(new))
    assert kda.kda_device_status() == 1
    want = [list(row) for row in table]
    want[1][2:4] = [free[count - 1], -1]
    want[2][1:3] = [free[count - 3], free[count - 4]]
    assert t.tolist() == want
    # its rows have no slots: sequence 1's from position 48 on
    slots = r.slots.tolist()
    assert all((s == -1) == (10 + 18 <= i < 30) for i, s in enumerate(slots))


@pytest.mark.parametrize("new", [[1] + [0] * 16382 + [1], [2 * (i % 997 == 5) + (i % 1009 == 7) for i in range(16384)],
                                 [0] * 3000 + [5] + [0] * 40 + [1, 0, 0, 1] + [0] * 500])
def test_rows_among_long_runs_of_sequences_without_any(new):
    lens = [(7 * i) % 40 for i in range(len(new))]
    need = sum(-(-(a + b) // 16) + (a // -16) for a, b in zip(lens, new))
    table, free, count, pages = pool(11, lens, 16, 4, need)
    check_reserve(table, lens, new, free, count, 16, pages, rows=sum(new) + 1)


def test_a_batch_goes_on_without_the_sequences_that_were_refused():
    """Prompts and tokens of more sequences than the pool has pages for, with no length read on the host:
    the rows that got places come first and are packed by what the lengths grew by; the others
    wait until pages come back."""
    N, Hk, H, D, page, width, scale = 5, 1, 2, 128, 16, 8, 128 ** -0.5
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [60, 50, 33, 20, 64]               # 4 + 4 + 3 + 2 + 4 pages
    q, k, v = (torch.randn((sum(lens), h, D), generator=g, device="cuda").to(torch.bfloat16) for h in (H, Hk, Hk))
    start = [0, 60, 110, 143, 163]
    cu_all = ints(start + [227])
    want = kda.kda_attn_fwd(q, k, v, scale, cu_seqlens=cu_all)
    cache = kda.kda_cache_alloc(12, Hk, page)  # sequences 0, 1 and 2 (11 pages), then none has room
    free, count = torch.randperm(12, generator=g, device="cuda").int(), ints([12])
    table, held, new = ints([[-1] * width] * N), ints([0] * N), ints(lens)

    def step(new, q, k, v):
        r = kda.kda_cache_reserve(table, held, new, free, count, page, rows=q.shape[0], new_free_count=count)
        cu = torch.nn.functional.pad((r.lens - held).cumsum(0, dtype=torch.int32), (1, 0))
        first = torch.argsort((r.slots < 0).byte(), stable=True)
        kda.kda_cache_append(cache, k[first], v[first], table, held, cu_seqlens=cu)
        out = torch.full_like(q, 7.0)
        kda.kda_cache_attn(cache, q[first], table, r.lens, scale, cu_seqlens=cu, out=out)
        return r, out[torch.argsort(first)]

    r, out = step(new, q, k, v)
    assert kda.kda_device_status() == 0
    assert r.lens.tolist() == [60, 50, 33, 0, 0] and count.item() == 1
    close = lambda a, b: (a.float() - b.float()).norm() < 8e-2 * b.float().norm()  # noqa: E731
    assert close(out[:143], want[:143]) and (out[143:] == 7).all()
    # the first two are done: their pages serve the others
    kda.kda_cache_release(table, r.lens, free, count, page, keep=ints([0, 0, 33, 0, 0]), new_free_count=count)
    held = r.lens * ints([0, 0, 1, 1, 1])
    r, out = step(ints([0, 0, 0, 20, 64]), q[143:], k[143:], v[143:])
    assert kda.kda_device_status() == 0
    assert r.lens.tolist() == [0, 0, 33, 20, 64] and close(out, want[143:]) and count.item() == 3
    used = [p for row, n in zip(table.tolist(), r.lens.tolist()) for p in row[: -(-n // page)]]
    assert sorted(used + free.tolist()[:3]) == list(range(12))
