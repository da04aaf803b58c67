"""A workspace in the wrong place, or one that does not hold its bytes at its pointer, is
refused before anything is launched."""
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda

i32 = torch.int32


def test_workspace():
    with pytest.raises(ValueError, match="device"):
        kda._space(torch.empty(1024, dtype=torch.uint8))
    for w in (torch.empty(1, dtype=torch.uint8).expand(1024), torch.empty(2048, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            kda._space(w)


def calls(w):
    """Each prefill with workspace w, of two tokens."""
    new = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    d, T = kda.dims(1), 2
    q, k, v, o = (new(T, 1, 128) for _ in range(4))
    pool, idx, cu = new(1, 1, 128, 128, t=torch.float32), new(1, t=i32), torch.tensor([0, T], dtype=i32, device="cuda")
    a, g = new(T, 1, t=torch.float32), new(T, 1, 128)
    beta = new(T, 1)
    scalar = kda.ScalarGate()
    yield lambda: kda.kda_prefill(d, kda.Gate(), q, k, v, g, beta, pool, idx, cu, 1, o, workspace=w)
    yield lambda: kda.kda_gdn_prefill(d, scalar, q, k, v, a, beta, pool, idx, cu, 1, o, workspace=w)
    yield lambda: kda.kda_lin_prefill(d, scalar, q, k, v, a, pool, idx, cu, 1, o, workspace=w)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(3))
def test_calls_refuse_it(i):
    size = 1 << 20
    for w in (torch.empty(size, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(size),
              torch.empty(2 * size, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            list(calls(w))[i]()
    list(calls(torch.empty(64 * size, dtype=torch.uint8, device="cuda")))[i]()
