"""Prefill of large tokens taken as they are, under decays that change much within 16 tokens:
what is computed on the way stays within FP32's range where the outputs do."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from tests import lin_util as lu
from tests.test_gpu_lin import SCALE, case, draw, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("decay", [-0.5, -3.0, -3.6, -5.0])
@pytest.mark.parametrize("size", [1e-4, 1.0, 1e4, 1e6])
def test_large_and_small_tokens(size, decay):
    c = case([200], H=1, HV=2, gate="given", norm=False)
    x = draw(c, 900)
    x["a"][:200] = decay
    for n in "qkv":
        x[n] = (x[n].float() * size).to(x[n].dtype)
    x["pool"] *= size ** 2
    o, pool = run(c, x)
    q, k, v = (lu.host(x[n]) for n in "qkv")
    g, S0 = lu.host(x["a"])[:200], lu.host(x["pool"])[int(x["idx"][0])]
    want, states = so.lin_sequence(S0, q, k, v, g, SCALE, False)
    o_bound, s_bound = lu.bounds(S0, q, k, v, g, SCALE, False, "bf16", exact_weights=True)
    lu.check("o", o, want, o_bound, "bf16")
    lu.check("state", pool[int(x["idx"][0])], states[-1], s_bound)
