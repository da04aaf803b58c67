"""Outputs of the linear-attention prefill are as exact as their own rounding: the bounds
of lin_util with weights and states taken whole, as decode's and verify's are."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from tests import lin_util as lu
from tests.test_gpu_lin import SCALE, case, draw, run

pytestmark = pytest.mark.gpu

CASES = [case([64]), case([63, 64, 65], H=2), case([333, 77], HV=4, gate="fixed", norm=False), case([257, 3], gate="out", H=2),
         case([190], gate="none", norm=False), case([2100], HV=2, gate="fixed"), case([130], gate="strong", dtype="f16"),
         case([190], gate="none", dtype="f16"), case([1000, 64, 5, 700], HV=2, gate="fixed", dtype="f16"),
         case([1537, 2, 640], H=2, gate="given", dtype="f16")]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_outputs_are_off_by_their_own_rounding(i):
    """An output's products with a state and with a chunk's weights are of two halves of the
    16-bit type, which leave 2^-17 of the magnitudes: within lin_util's 2^-14 for all that is
    not the output's own rounding.  (Rounded once, they leave 2^-8 or 2^-11 of them.)"""
    c = CASES[i]
    x = draw(c, 500 + i)
    o, pool = run(c, x)
    g = so.lin_decay(len(x["q"]), lu.host(x["a"]), lu.host(x["A_log"]), lu.host(x["dt_bias"]))
    states = lu.host(x["pool"])
    for n, slot in enumerate(x["idx"].tolist()):
        s = slice(int(x["cu"][n]), int(x["cu"][n + 1]))
        q, k, v = (lu.host(x[name][s]) for name in "qkv")
        want, _ = so.lin_sequence(states[slot], q, k, v, g[s], SCALE, c["norm"])
        bound, _ = lu.bounds(states[slot], q, k, v, g[s], SCALE, c["norm"], c["dtype"], exact_weights=True)
        lu.check(f"o of sequence {n}", o[s], want, bound, c["dtype"])
        # all together: the outputs' rounding in the oracle, and 2^-14 of the RMS
        rounded = torch.tensor(want).to(lu.DT[c["dtype"]]).double().numpy()
        off, least = (np.sqrt(np.mean((y - want) ** 2)) for y in (o[s].double().cpu().numpy(), rounded))
        assert off <= least + 2.0 ** -14 * np.sqrt(np.mean(want ** 2)), f"{off:.3g} RMS off, {least:.3g} by the rounding"
