"""Pages kept in 8 or 4 bits and read back: codes, scales and values are exact, so
every comparison is of equal bits."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu
K = 128
i32 = torch.int32


def archive(slots, layers, rows, bits, fill=None):
    codes = torch.zeros(slots, layers, rows, K if bits == 8 else K // 2, dtype=torch.int8 if bits == 8 else torch.uint8, device="cuda")
    scales = torch.zeros(slots, layers, rows, 1 if bits == 8 else 4, device="cuda")
    if fill is not None:
        codes.fill_(fill)
        scales.fill_(fill)
    return codes, scales


def unpack(codes, bits):
    c = codes.cpu().numpy()
    if bits == 8:
        return c
    lo, hi = (c & 15).astype(np.int8), (c >> 4).astype(np.int8)
    both = np.stack([lo, hi], -1).reshape(*c.shape[:-1], K)
    return np.where(both > 7, both - 16, both).astype(np.int8)


def lst(*x):
    return torch.tensor(x, dtype=i32, device="cuda")


def same(a, b):
    """Equal bits, NaN as NaN."""
    a, b = np.asarray(a), np.asarray(b)
    return np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


def kinds(shape, seed):
    """Values of every kind: usual rows, zeros, a single value, ties, tiny, huge and
    uneven ones, not finite ones."""
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape).astype(np.float32) * np.exp(g.standard_normal(shape[:-1] + (1,)) * 3).astype(np.float32)
    flat = x.reshape(-1, K)
    n = len(flat)
    for i in range(n):
        kind = i % 12
        if kind == 1:
            flat[i] = 0
        elif kind == 2:
            flat[i] = 0
            flat[i, i % K] = -3.7
        elif kind == 3:  # whole and half steps of a scale of 2^-k
            flat[i] = (g.integers(-254, 255, K) / 2 * 2.0 ** -(i % 40)).astype(np.float32)
            flat[i, 5] = 127 * 2.0 ** -(i % 40)
        elif kind == 4:
            flat[i] *= np.float32(1e-38)
        elif kind == 5:
            flat[i] = g.integers(-300, 300, K) * np.float32(1e-45)
        elif kind == 6:
            flat[i] = np.clip(flat[i].astype(np.float64) * 1e36, -3e38, 3e38)
        elif kind == 7:  # halves of a scale that is no power of two
            s = np.float32(g.uniform(0.5, 2))
            flat[i] = (g.integers(-127, 127, K) + 0.5).astype(np.float32) * s
            flat[i, 9] = 127 * s
        elif kind == 8 and i % 24 == 8:
            flat[i, 40] = np.nan
        elif kind == 9 and i % 36 == 9:
            flat[i, 127] = -np.inf
        elif kind == 10:
            flat[i] = np.float32(3.4e38) * g.uniform(-1, 1, K).astype(np.float32)
    return x


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("layers,rows", [(1, 1), (2, 63), (3, 64), (1, 65), (2, 512)])
def test_store_and_load(bits, layers, rows):
    slots, keep = 5, 4
    x = kinds((layers, slots, rows, K), rows)
    pool = torch.from_numpy(x).cuda()
    codes, scales = archive(keep, layers, rows, bits, fill=3)
    err = torch.zeros(1, dtype=i32, device="cuda")
    kda.kda_pool_store(pool, codes, scales, lst(4, 0, -1, 2, 4), lst(1, 3, 0, -1, 2), err_flag=err)
    assert err.item() == 0 and same(pool.cpu().numpy(), x)
    want_c, want_s, want_v = so.archived(x[:, [4, 0]].reshape(-1, K), bits)
    shape = (layers, 2, rows)
    want_c, want_s, want_v = want_c.reshape(*shape, K), want_s.reshape(*shape, -1), want_v.reshape(*shape, K)
    got_c, got_s = unpack(codes, bits), scales.cpu().numpy()
    for i, at in ((0, 1), (1, 3), (0, 2)):
        assert same(got_c[at], want_c[:, i]) and same(got_s[at], want_s[:, i])
    assert (codes[0] == 3).all() and (scales[0] == 3).all()
    kda.kda_pool_load(codes, scales, pool, lst(3, 1, -1, 2), lst(1, 0, 3, -1), err_flag=err)
    assert err.item() == 0
    got = pool.cpu().numpy()
    assert same(got[:, 1], want_v[:, 1]) and same(got[:, 0], want_v[:, 0])
    assert same(got[:, 2:], x[:, 2:])


@pytest.mark.parametrize("bits", [8, 4])
def test_within_half_a_scale(bits):
    x = torch.randn(1, 2, 8, K, device="cuda")
    codes, scales = archive(1, 1, 8, bits)
    kda.kda_pool_store(x, codes, scales, lst(0), lst(0))
    kda.kda_pool_load(codes, scales, x, lst(0), lst(1))
    unit = scales[0].repeat_interleave(K // scales.shape[-1], -1)
    # half a scale, and the FP32 rounding of the value read back
    assert ((x[:, 0] - x[:, 1]).abs() <= unit * 0.5 + x[:, 1].abs() * 2.0 ** -24).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_bad_pairs_are_flagged_and_left_out(bits):
    x = torch.randn(2, 4, 3, K, device="cuda")
    for src, dst, good in (((0, 4), (0, 1), [0]), ((0, -2), (0, 1), [0]), ((1, 2), (0, 5), [0]), ((1, 2), (-3, 1), [1]),
                           ((0, 1, 2), (2, 2, 1), [2])):
        codes, scales = archive(3, 2, 3, bits, fill=3)
        before = codes.clone()
        err = torch.zeros(1, dtype=i32, device="cuda")
        kda.kda_pool_store(x, codes, scales, lst(*src), lst(*dst), err_flag=err)
        assert err.item() == kda.KDA_DEVERR_PAGE
        written = {dst[i] for i in good}
        for s in range(3):
            assert torch.equal(codes[s], before[s]) == (s not in written)
    codes, scales = archive(3, 2, 3, bits)
    kda.kda_pool_store(x, codes, scales, lst(0, 1, 2), lst(0, 1, 2))
    for src, dst, good in (((0, 3), (0, 1), [0]), ((1, 2), (4, 1), [1]), ((0, 1, 2), (3, 3, 0), [2])):
        pool = x.clone()
        err = torch.zeros(1, dtype=i32, device="cuda")
        kda.kda_pool_load(codes, scales, pool, lst(*src), lst(*dst), err_flag=err)
        assert err.item() == kda.KDA_DEVERR_PAGE
        written = {dst[i] for i in good}
        for s in range(4):
            assert torch.equal(pool[:, s], x[:, s]) == (s not in written)


@pytest.mark.parametrize("bits", [8, 4])
def test_layers_apart_and_capture(bits):
    """Layers further apart than their slots take, lists that change between
    replays."""
    big = torch.randn(2, 9, 4, 128, K, device="cuda")
    pool = big[:, 2:6]
    codes, scales = archive(4, 2, 512, bits)
    src, dst, back = lst(0, 3), lst(2, 1), lst(1, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_pool_store(pool, codes, scales, src, dst)
        kda.kda_pool_load(codes, scales, pool, dst, back)
    for s, d, b in (((0, 3), (2, 1), (1, 2)), ((2, -1), (0, 3), (3, 0))):
        src.copy_(lst(*s)), dst.copy_(lst(*d)), back.copy_(lst(*b))
        big.normal_()
        codes.zero_(), scales.zero_()
        x = big.clone()
        graph.replay()
        for i in range(2):
            page = x[:, 2 + s[i]].cpu().numpy()
            want = so.archived(page.reshape(-1, K), bits)[2].reshape(page.shape) if s[i] >= 0 else np.zeros_like(page)
            assert same(big[:, 2 + b[i]].cpu().numpy(), want)
        rest = [j for j in range(9) if j - 2 not in b]
        assert torch.equal(big[:, rest], x[:, rest])
