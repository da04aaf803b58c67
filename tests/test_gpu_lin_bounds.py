"""Prefill with cu_seqlens that are not bounds throughout: which sequences run, what those
get, and that nothing else is written."""
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so
from tests import lin_util as lu
from tests.test_gpu_lin import SCALE, case, draw, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cu,runs", [
    ([0, 50, 130, 120], [0]),  # past the last token, and back
    ([1, 50, 60, 120], [1, 2]),  # the first does not start at 0
    ([0, 50, 60, 119], [0, 1]),  # the last does not end at the last token
    ([0, -4, 60, 120], [2]),
    ([0, 50, 50, 120], [0, 2]),  # one without tokens: no error
    ([0, 50, 40, 120], []),  # sequences that overlap have more tokens than there are: none runs
])
def test_sequences_with_bounds_of_their_own(cu, runs, dtype):
    c = case([50, 10, 60], H=1, HV=2, dtype=dtype)
    x = dict(draw(c, 950), cu=torch.tensor(cu, dtype=torch.int32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, pool = run(c, x, err_flag=err)
    assert err.item() == (0 if cu == sorted(cu) and cu[0] == 0 and cu[-1] == 120 else kda.KDA_DEVERR_SEQLENS)
    g = so.lin_decay(len(x["q"]), lu.host(x["a"]), lu.host(x["A_log"]), lu.host(x["dt_bias"]))
    left, slots = torch.ones(120, dtype=torch.bool), set(range(len(pool)))
    for n in runs:
        s, slot = slice(cu[n], cu[n + 1]), int(x["idx"][n])
        q, k, v = (lu.host(x[name][s]) for name in "qkv")
        S0 = lu.host(x["pool"])[slot]
        want, states = so.lin_sequence(S0, q, k, v, g[s], SCALE, True)
        o_bound, s_bound = lu.bounds(S0, q, k, v, g[s], SCALE, True, dtype, exact_weights=True)
        lu.check(f"o of sequence {n}", o[s], want, o_bound, dtype)
        lu.check(f"state of sequence {n}", pool[slot], states[-1], s_bound)
        left[s] = False
        slots.discard(slot)
    assert (o[left.cuda()] == 7).all(), "an output of no sequence"
    rest = sorted(slots)
    assert torch.equal(pool[rest].cpu(), x["pool"][rest]), "a slot of no sequence that runs"
