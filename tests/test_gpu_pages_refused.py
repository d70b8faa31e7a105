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
