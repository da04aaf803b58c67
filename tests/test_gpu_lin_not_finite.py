"""A value that is not finite stays in its rows of the state, however a sequence is cut and
whatever its decays leave: a state has the same such entries as token by token."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so
from tests import lin_util as lu
from tests.test_gpu_lin import SCALE, case, draw, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("length,HV,decay", [(2100, 1, -2.0), (2100, 1, -0.001), (5000, 2, -0.5), (9000, 1, -1.0), (100, 1, -2.0)])
def test_bad_values_outlive_their_decay(length, HV, decay, dtype):
    c = case([length], H=1, HV=HV, dtype=dtype, gate="given")
    assert length == 100 or kda.kda_lin_prefill_workspace_size(lu.dims(c), 1, length) > 0, "in several segments"
    x = draw(c, 800)
    x["a"][:length] = decay
    x["v"][70, 0, 5] = float("nan")
    x["v"][length // 2, 0, 9] = float("inf")
    x["pool"][int(x["idx"][0]), HV - 1, 17, 3] = float("-inf")
    x["pool"][int(x["idx"][0]), HV - 1, 18, 4] = float("nan")
    o, pool = run(c, x)
    q, k, v = (lu.host(x[n]) for n in "qkv")
    with np.errstate(invalid="ignore"):
        want, states = so.lin_sequence(lu.host(x["pool"])[int(x["idx"][0])], q, k, v, lu.host(x["a"])[:length], SCALE, True)
    bad = ~np.isfinite(states[-1])
    assert bad[0, 5].all() and bad[0, 9].all() and bad[HV - 1, 17, 3] and bad[HV - 1, 18, 4]
    assert not (~np.isfinite(pool[int(x["idx"][0])].cpu().numpy()) ^ bad).any()
    # outputs: the same from the next chunk on
    bad, got = ~np.isfinite(want), ~np.isfinite(o.float().cpu().numpy())
    for t in range(0, length, 64):
        if not any(t <= at < t + 64 for at in (70, length // 2)):
            assert not (got[t:t + 64] ^ bad[t:t + 64]).any(), f"tokens from {t}"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("decay", [None, -0.01])
def test_a_bad_key_leaves_the_rest_of_its_chunk(dtype, bad, decay):
    """Keys as they are: one channel of one key is not finite.  The tokens before it, and the
    state's other channels, are what they are without it."""
    c = case([190], H=1, HV=2, dtype=dtype, gate="given", norm=False)
    x = draw(c, 810)
    if decay is not None:  # a state that keeps the chunk
        x["a"][:190] = decay
    x["k"][70, 0, 3] = bad
    o, pool = run(c, x)
    q, k, v = (lu.host(x[n]) for n in "qkv")
    k[70, 0, 3] = 0
    S0, g = lu.host(x["pool"])[int(x["idx"][0])], lu.host(x["a"])[:190]
    want, states = so.lin_sequence(S0, q, k, v, g, SCALE, False)
    k[70, 0, 3] = 65504  # FP16's largest, by which its chunk's powers of two go
    o_bound, _ = lu.bounds(S0, q, k, v, g, SCALE, False, dtype)
    o_bound[64:70] += 2.0 ** -39 * SCALE * np.sqrt((q[64:70] ** 2).sum(-1))[:, :, None] * 65504 * 128 ** 0.5 * np.cumsum(np.abs(v[64:70]), 0)
    lu.check("o before it", o[:70], want[:70], o_bound[:70], dtype)
    k[70, 0, 3] = 0
    _, s_bound = lu.bounds(S0, q, k, v, g, SCALE, False, dtype, exact_weights=True)
    # FP16 parts end 2^-39 below the chunk's largest key, here at most 65504 sqrt 128 times its decay
    s_bound = s_bound + (2.0 ** -39 * 65504 * 128 ** 0.5 * np.abs(v[64:128]).sum(0)[:, :, None] if dtype == "f16" else 0)
    state = pool[int(x["idx"][0])].cpu()
    assert not torch.isfinite(state[:, :, 3]).any()
    rest = [i for i in range(128) if i != 3]
    lu.check("state", state[:, :, rest], states[-1][:, :, rest], s_bound[:, :, rest])
