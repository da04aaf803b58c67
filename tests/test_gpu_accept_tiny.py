"""Rows whose weights are at the lower end of their type, or of very different
size: against whole numbers of the smallest weight."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda

pytestmark = pytest.mark.gpu


def draw(p, q, u, V, pad):
    """Next token behind p (rows V + pad apart); q: a draft whose token falls."""
    T = 1 if q is None else 2
    target = torch.zeros(1, T, V + pad, dtype=p.dtype)
    target[0, 0, :V] = p
    out = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    tokens = torch.tensor([[0, 3][:T]], dtype=torch.int32, device="cuda")
    draft = None if q is None else torch.cat([q, q.new_zeros(pad)]).view(1, 1, -1).cuda()[..., :V]
    kda.kda_accept_chain(target.cuda()[..., :V], draft, tokens, torch.full((1, T), u, device="cuda"), *out)
    assert int(out[0]) == 0
    return int(out[1])


def want(units, u):
    """units: whole numbers; the lowest j whose running sum exceeds u times the whole."""
    num, den = float(u).as_integer_ratio()
    run, whole = 0, sum(units)
    for j, x in enumerate(units):
        run += x
        if x and run * den > num * whole:
            return j
    return max(j for j, x in enumerate(units) if x)


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("V", [8, 4000])
@pytest.mark.parametrize("exponent", [-149, -140, -133, -124, -80, -61, -20])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tiny_weights(dtype, exponent, V, pad):
    if dtype is torch.bfloat16 and exponent < -133:
        pytest.skip("below the type's smallest number")
    rng = np.random.default_rng(V - exponent)
    for n in (3, 5, V):
        units = np.zeros(V, np.int64)
        units[rng.permutation(V)[:n]] = rng.integers(1, 4, n)
        p = torch.from_numpy(units * 2.0 ** exponent).to(dtype)
        assert torch.equal(p.double() * 2.0 ** -exponent, torch.from_numpy(units).double())
        for u in (0.0, 0.4, 0.5, 0.6, 0.999, *rng.random(5)):
            u = float(np.float32(u))
            assert draw(p, None, u, V, pad) == want(units.tolist(), u), (n, u)


@pytest.mark.parametrize("pad", [0, 1])
def test_tiny_remainders(pad):
    """p and q are the same but for some weights of a few times 2^-149."""
    V = 4000
    rng = np.random.default_rng(1)
    base = torch.softmax(torch.from_numpy(rng.normal(size=V)), 0).float()
    base[::7] = 0.0
    base[3] = 0.0
    units = np.zeros(V, np.int64)
    units[7 * rng.permutation(V // 7)[:5]] = rng.integers(1, 4, 5)
    p = base + torch.from_numpy(units * 2.0 ** -149).float()
    for u in (0.3, 0.5, 0.6, *rng.random(6)):
        u = float(np.float32(u))
        assert draw(p, base, u, V, pad) == want(units.tolist(), u), u
