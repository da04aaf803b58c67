"""Fork into rows that hold neither a slot nor -1: refused, and left as they are."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("value", [-2, -3, -7, -1000, 8, 1 << 30])
@pytest.mark.parametrize("rows", [[2], [2, 3], [3, 2], [2, 2, 3], [3, 3, 2], [4, 3, 5, 2, 6]])
def test_rows_out_of_range_are_refused(value, rows):
    rng = np.random.default_rng(0)
    pool = rng.normal(size=(2, 8, 12)).astype(np.float32)
    table = np.array([5, 1, value, -1, -1, -1, -1], np.int32)
    used = np.zeros(8, np.uint8)
    used[[5, 1]] = 1
    d_pool, d_used, d_table = (torch.from_numpy(x.copy()).cuda() for x in (pool, used, table))
    err = i32([0])
    kids = kda.kda_pool_fork(d_pool, d_used, d_table, i32([0] * len(rows)), i32(rows), err_flag=err)
    assert so.pool_fork(pool, used, table, [0] * len(rows), rows) >= 1
    assert table[2] == value and int(err) == kda.KDA_DEVERR_PAGE
    assert np.array_equal(d_table.cpu().numpy(), table) and np.array_equal(d_used.cpu().numpy(), used)
    assert np.array_equal(d_pool.cpu().numpy(), pool)
    first = [rows.index(r) == i and r != 2 for i, r in enumerate(rows)]
    assert kids.tolist() == [int(table[r]) if f else -1 for r, f in zip(rows, first)]
