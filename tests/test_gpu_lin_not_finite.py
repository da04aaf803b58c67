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
