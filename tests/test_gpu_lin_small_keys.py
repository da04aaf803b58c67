"""FP16 prefill of keys taken as they are: states are as exact as those of larger or
normalised keys, however small the keys of a chunk are."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from tests import lin_util as lu
from tests.test_gpu_lin import SCALE, case, draw, run

pytestmark = pytest.mark.gpu


def check(c, x):
    """Bounds of lin_util without its 2^-25 a token for the parts of an FP16 key: a chunk's
    decayed keys are taken times a power of two that brings the largest above 2^14, so that the
    steps of 2^-24 at the parts' end are 2^-38 of it, and 2^-22 of a key whose parts are whole:
    far below 2^-14 of the magnitudes' sum.

    A row's weights in a chunk are taken times a power of two that brings |q_i| max_j |k_j| above
    2^14 (that of all the chunk's keys, whatever the decays leave of them), and their parts end at
    steps of 2^-24 too: each weight is off by up to 2^-25 / 2^14 = 2^-39 of that product, and the
    output by scale 2^-39 |q_i| max_j |k_j| sum_j |v_j|, as lin_util states it for weights
    rounded once."""
    o, pool = run(c, x)
    g = so.lin_decay(len(x["q"]), lu.host(x["a"]), lu.host(x["A_log"]), lu.host(x["dt_bias"]))
    states = lu.host(x["pool"])
    for n, slot in enumerate(x["idx"].tolist()):
        s = slice(int(x["cu"][n]), int(x["cu"][n + 1]))
        q, k, v = (lu.host(x[name][s]) for name in "qkv")
        want, after = so.lin_sequence(states[slot], q, k, v, g[s], SCALE, c["norm"])
        o_bound, s_bound = lu.bounds(states[slot], q, k, v, g[s], SCALE, c["norm"], "f16", exact_weights=True)
        lu.check(f"state of sequence {n}", pool[slot], after[-1], s_bound)
        norm_of = lambda y: np.repeat(np.sqrt((y * y).sum(-1)), v.shape[1] // q.shape[1], 1)  # noqa: E731
        for t in range(0, len(q), 64):
            part = slice(t, t + 64)
            o_bound[part] += 2.0 ** -39 * SCALE * (norm_of(q[part]) * norm_of(k[part]).max(0))[:, :, None] * np.cumsum(np.abs(v[part]), 0)
        lu.check(f"o of sequence {n}", o[s], want, o_bound, "f16")


@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("lengths", [[5, 64, 200], [1500]])
def test_small_keys(size, lengths):
    c = case(lengths, H=1, HV=2, dtype="f16", gate="fixed", norm=False)
    x = draw(c, 700)
    x["k"] = (x["k"].float() * size).half()
    x["pool"] = x["pool"] * 0  # nothing larger beside them
    check(c, x)


def test_keys_of_many_sizes():
    """Large keys that the chunk's decays leave nothing of, before small ones; chunks of zeros;
    FP16's smallest and largest numbers."""
    c = case([64, 192, 30, 64, 64], H=1, HV=2, dtype="f16", gate="given", norm=False)
    x = draw(c, 701)
    x["pool"] = x["pool"] * 0
    k = x["k"].float()
    x["a"][:] = -0.01
    x["a"][:64] = -3.0
    k[:16] *= 1000
    k[16:64] *= 1e-3
    k[64:128] = 0
    k[128:192] *= 1e-4
    k[192:256] = 0
    k[256:286] = 0
    k[286:350] = k[286:350].sign() * 2.0 ** -24
    k[350:] = k[350:].sign() * 65504
    x["k"] = k.half()
    x["v"][350:] *= 0.1
    x["q"][350:] *= 1e-4  # (outputs within FP16's range)
    check(c, x)
