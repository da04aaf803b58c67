"""Compact and fork of pools around the size at which a map of the used slots
outgrows a kernel's 48 KiB of shared memory, and of the largest one."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def make(slots, rows=300):
    """16-byte pages; the used ones at both ends and between."""
    rng = np.random.default_rng(slots)
    at = np.unique(np.concatenate([[0, 5, slots - 1, slots - 2], rng.integers(0, slots, rows)]))
    rng.shuffle(at)
    table = np.concatenate([at, [-1] * 20]).astype(np.int32)
    used = np.zeros(slots, np.uint8)
    used[at] = 1
    return rng, rng.normal(size=(1, slots, 4)).astype(np.float32), used, table


def same(dev, host):
    return np.array_equal(dev.cpu().numpy(), host)


# 48 KiB is 196576 slots of map alone; the kernels' own arrays take some of it
@pytest.mark.parametrize("slots", [192480, 192481, 195520, 195521, 196000, 196032, 196033, 196300, 196576, 196577, 196608,
                                   1 << 19])
def test_maps_of_any_size(slots):
    rng, pool, used, table = make(slots)
    d_pool, d_used, d_table = (torch.from_numpy(x.copy()).cuda() for x in (pool, used, table))
    count, err = i32([-1]), i32([0])
    rows = list(range(len(table) - 20, len(table)))
    parents = [int(x) for x in rng.integers(-1, len(table) - 20, 20)]
    assert so.pool_fork(pool, used, table, parents, rows) == 0  # into the holes
    kda.kda_pool_fork(d_pool, d_used, d_table, i32(parents), i32(rows), err_flag=err)
    assert same(d_pool, pool) and same(d_used, used) and same(d_table, table)
    want = so.pool_compact(pool, used, table)
    kda.kda_pool_compact(d_pool, d_used, d_table, count, err_flag=err)
    assert int(count) == want and int(err) == 0
    assert same(d_pool, pool) and same(d_used, used) and same(d_table, table)


def test_the_largest_pool_in_a_graph():
    slots = 1 << 19
    _, pool, used, table = make(slots)
    first = [torch.from_numpy(x.copy()).cuda() for x in (pool, used, table)]
    count = i32([-1])
    kda.kda_pool_compact(*first, count)  # before capture
    d_pool, d_used, d_table = (torch.from_numpy(x.copy()).cuda() for x in (pool, used, table))
    parents, rows, kids = i32([3, -1]), i32([len(table) - 1, len(table) - 2]), i32([0, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_pool_compact(d_pool, d_used, d_table, count)
        kda.kda_pool_fork(d_pool, d_used, d_table, parents, rows, children=kids)
    graph.replay()
    so.pool_compact(pool, used, table)
    so.pool_fork(pool, used, table, [3, -1], [len(table) - 1, len(table) - 2])
    assert same(d_pool, pool) and same(d_used, used) and same(d_table, table)
    assert kids.tolist() == table[[-1, -2]].tolist()
