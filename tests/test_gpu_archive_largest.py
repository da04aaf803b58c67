"""Pages that hold FP32's largest numbers come back finite, within half a scale."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from tests.test_gpu_archive import K, archive, lst

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 4])
def test_largest_numbers(bits):
    rows, group = 256, 128 if bits == 8 else 32
    big = np.float32(np.finfo(np.float32).max)
    x = np.random.default_rng(3).uniform(-1, 1, (rows, K)).astype(np.float32) * big
    at = big
    for i in range(0, rows, 2):  # the largest number, and one after the other below it, of either sign
        x[i, (7 * i) % K] = at if i % 4 else -at
        at = np.nextafter(at, np.float32(0))
    pool = torch.zeros(1, 2, 1, rows, K, device="cuda")
    pool[0, 0, 0] = torch.tensor(x)
    codes, scales = archive(1, 1, rows, bits)
    kda.kda_pool_store(pool, codes, scales, lst(0), lst(0))
    kda.kda_pool_load(codes, scales, pool, lst(0), lst(1))
    back, s = pool[0, 1, 0].cpu().numpy().astype(np.float64), scales.cpu().numpy().astype(np.float64).reshape(-1, 1)
    assert np.isfinite(back).all()
    # half a scale; FP32's rounding of the value, half a step of the largest, 2^103; and the scale's
    # own, 2^-24 of a value, which moves a quotient at a half to the other code
    off = np.abs(back - x.astype(np.float64)).reshape(-1, group)
    assert (off <= s / 2 + 2.0 ** 103 + 2.0 ** -24 * float(big)).all()
