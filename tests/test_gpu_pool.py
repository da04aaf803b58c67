"""Pages of a state pool against the plain oracle: bit for bit."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def make(seed, layers, slots, page, rows):
    rng = np.random.default_rng(seed)
    pool = torch.from_numpy(rng.normal(size=(layers, slots, page)).astype(np.float32))
    table = np.full(rows + 2, -1, np.int32)
    table[:rows] = rng.permutation(slots)[:rows]
    used = np.zeros(slots, np.uint8)
    used[table[:rows]] = 1
    return rng, pool, used, table


SHAPES = [(1, 1, 4, 1), (1, 2, 4, 1), (2, 16, 100, 6), (1, 33, 4, 20), (3, 240, 260, 150), (1, 1000, 8, 700),
          (1, 40000, 4, 30000)]


@pytest.mark.parametrize("layers,slots,page,rows", SHAPES)
def test_turnover(layers, slots, page, rows):
    """Free, compact, fork, twice over."""
    rng, pool, used, table = make(slots, layers, slots, page, rows)
    d_pool, d_used, d_table = pool.cuda(), torch.from_numpy(used).cuda(), torch.from_numpy(table).cuda()
    count, err = i32([-1]), i32([0])
    ref = pool.numpy().copy()
    for _ in range(2):
        gone = rng.permutation(rows)[:max(1, rows // 3)].astype(np.int32)
        so.pool_free(used, table, gone)
        kda.kda_pool_free(d_used, d_table, i32(gone), err_flag=err)
        assert np.array_equal(d_used.cpu().numpy(), used) and np.array_equal(d_table.cpu().numpy(), table)
        want = so.pool_compact(ref, used, table)
        kda.kda_pool_compact(d_pool, d_used, d_table, count, err_flag=err)
        assert int(count) == want
        assert np.array_equal(d_used.cpu().numpy(), used) and np.array_equal(d_table.cpu().numpy(), table)
        assert np.array_equal(d_pool.cpu().numpy(), ref)
        stay = [r for r in range(rows) if table[r] >= 0]
        parents = np.array([int(rng.choice(stay + [-1])) for _ in gone], np.int32)
        assert so.pool_fork(ref, used, table, parents, gone) == 0
        kda.kda_pool_fork(d_pool, d_used, d_table, i32(parents), i32(gone), err_flag=err)
        assert np.array_equal(d_used.cpu().numpy(), used) and np.array_equal(d_table.cpu().numpy(), table)
        assert np.array_equal(d_pool.cpu().numpy(), ref)
    assert int(err) == 0


def test_compact_of_full_empty_and_reversed_pools():
    for used in ([1, 1, 1, 1], [0, 0, 0, 0], [0, 0, 1, 1], [0, 1, 0, 1, 1]):
        used = np.array(used, np.uint8)
        table = np.array([s for s in range(len(used)) if used[s]] + [-1], np.int32)
        pool = np.arange(len(used) * 4, dtype=np.float32).reshape(1, len(used), 4)
        dp, du, dt, count = torch.from_numpy(pool.copy()).cuda(), torch.from_numpy(used.copy()).cuda(), torch.from_numpy(
            table.copy()).cuda(), i32([-1])
        kda.kda_pool_compact(dp, du, dt, count)
        assert int(count) == so.pool_compact(pool, used, table)
        assert np.array_equal(dp.cpu().numpy(), pool) and np.array_equal(dt.cpu().numpy(), table)
        assert np.array_equal(du.cpu().numpy(), used)


def test_fork_refusals_and_a_full_pool():
    """Duplicate rows, rows that hold a page, parents without one, parents that
    only get theirs in this call, and more forks than free pages."""
    _, pool, used, table = make(3, 2, 8, 12, 5)
    cases = [([0, 1], [5, 5]), ([0], [1]), ([6], [5]), ([0, 5], [5, 6]), ([0, -1, 1, -1], [5, -1, 6, 6]), ([9], [5]),
             ([0], [77])]
    for parents, rows in cases:
        err = i32([0])
        dp, du, dt = pool.cuda(), torch.from_numpy(used).cuda(), torch.from_numpy(table).cuda()
        kda.kda_pool_fork(dp, du, dt, i32(parents), i32(rows), err_flag=err)
        rp, ru, rt = pool.numpy().copy(), used.copy(), table.copy()
        inside = [(p, r) for p, r in zip(parents, rows) if p < len(table) and r < len(table)]
        so.pool_fork(rp, ru, rt, [p for p, _ in inside], [r for _, r in inside])
        assert int(err) == kda.KDA_DEVERR_PAGE
        assert np.array_equal(du.cpu().numpy(), ru) and np.array_equal(dt.cpu().numpy(), rt)
        assert np.array_equal(dp.cpu().numpy(), rp)
    wide = np.concatenate([table, np.full(6, -1, np.int32)])
    rows = list(range(5, 13))
    err = i32([0])
    dp, du, dt = pool.cuda(), torch.from_numpy(used).cuda(), torch.from_numpy(wide).cuda()
    kda.kda_pool_fork(dp, du, dt, i32([0] * 8), i32(rows), err_flag=err)
    rp, ru, rt = pool.numpy().copy(), used.copy(), wide.copy()
    assert so.pool_fork(rp, ru, rt, [0] * 8, rows) == 5
    assert int(err) == kda.KDA_DEVERR_POOL_FULL
    assert np.array_equal(dt.cpu().numpy(), rt) and np.array_equal(dp.cpu().numpy(), rp)


def test_free_refusals():
    used = torch.tensor([1, 0, 1, 1, 1], dtype=torch.uint8).cuda()
    table = i32([0, 1, 2, 9, -1])
    err = i32([0])
    kda.kda_pool_free(used, table, i32([0, 0, -1, 4]), err_flag=err)  # twice: freed once; nothing to free
    assert int(err) == 0 and table.tolist() == [-1, 1, 2, 9, -1] and used.tolist() == [0, 0, 1, 1, 1]
    for row in (1, 3, 5, -2):  # a page not in use, a slot and rows out of range
        err.zero_()
        kda.kda_pool_free(used, table, i32([row]), err_flag=err)
        assert int(err) == kda.KDA_DEVERR_PAGE
    assert used.tolist() == [0, 0, 1, 1, 1]


@pytest.mark.parametrize("page", [4, 1000, 16384 + 4])
def test_copy(page):
    pool = torch.randn(2, 9, page).cuda()
    before = pool.clone()
    err = i32([0])
    kda.kda_pool_copy(pool, i32([0, 3, -1, 0, 8]), i32([1, 2, 5, -1, 7]), err_flag=err)
    want = before.clone()
    want[:, 1], want[:, 2], want[:, 7] = before[:, 0], before[:, 3], before[:, 8]
    assert int(err) == 0 and torch.equal(pool, want)
    # a swap, two copies into one page, slots out of range: refused, the rest is copied
    kda.kda_pool_copy(pool, i32([0, 1, 2, 3, 9, 4]), i32([1, 0, 5, 5, 6, 8]), err_flag=err)
    want[:, 8] = want[:, 4]
    assert int(err) == kda.KDA_DEVERR_PAGE and torch.equal(pool, want)


def test_layers_further_apart_and_offsets_past_32_bits():
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB")
    base = torch.zeros(2, 2200, 1 << 18, dtype=torch.float32, device="cuda")  # 1 MiB pages, 2.3 GB a layer
    pool = base[:, 50:2150]
    pool[:, 2098] = 5.0
    kda.kda_pool_copy(pool, i32([2098]), i32([2099]))
    assert bool((pool[:, 2099] == 5).all()) and bool((base[:, 2150:] == 0).all()) and bool((pool[:, 2097] == 0).all())
