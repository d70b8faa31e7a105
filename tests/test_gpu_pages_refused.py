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
