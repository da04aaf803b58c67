"""Sums of long rows.  Weights are whole multiples of 2^-45, so every border is
known exactly; u = 1/2 puts the goal a few multiples below a border, where a sum
that loses its low bits draws the wrong token."""
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda

pytestmark = pytest.mark.gpu
BIG, X = 1 << 44, 3 * (1 << 21) + (1 << 19) + 1  # each X leaves 2^19 + 1 behind where a sum of BIG is rounded to 24 bits


def whole_parts(n):
    """n as whole numbers of 24 bits at most."""
    out = []
    while n:
        shift = max(n.bit_length() - 24, 0)
        out.append(n >> shift << shift)
        n -= out[-1]
    return out


def row(V, first, below):
    """Weights BIG, X, X, .. at `first`; behind them what makes half of the whole
    their sum less `below`.  Returns the row and the first token behind."""
    sum_first = BIG + X * (len(first) - 1)
    p = torch.zeros(V, dtype=torch.float64)
    p[first] = float(X)
    p[first[0]] = float(BIG)
    rest = whole_parts(sum_first - 2 * below)
    at = V // 2 + 1000 * torch.arange(len(rest))
    p[at] = torch.tensor([float(x) for x in rest], dtype=torch.float64)
    p32 = (p * 2.0 ** -45).float()
    assert torch.equal(p32.double() * 2.0 ** 45, p)
    return p32, int(at[0])


def draw(p, q=None, token=0, offset=0):
    V = p.numel()
    T = 1 if q is None else 2
    buf = torch.zeros(offset + T * V, device="cuda")
    target = buf[offset:].view(1, T, V)
    target[0, 0] = p.cuda()
    out = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    tokens = torch.tensor([[0, token][:T]], dtype=torch.int32, device="cuda")
    kda.kda_accept_chain(target, None if q is None else q.cuda().view(1, 1, V), tokens, torch.full((1, T), 0.5, device="cuda"),
                         *out)
    assert int(out[0]) == 0
    return int(out[1])


@pytest.mark.parametrize("offset", [0, 1])  # rows on 16 bytes, and not
@pytest.mark.parametrize("log_v", [16, 20, 24, 26])
def test_sums_keep_their_low_bits(log_v, offset):
    V = 1 << log_v
    j = torch.arange(V // 1024)  # one lane's entries of the first block
    first = j[j % 32 == 0] if offset else j[(j % 128 == 0) | (j % 128 == 2)]
    if V == 1 << 16:
        first = torch.arange(1024)
    p, behind = row(V, first, 10)
    assert draw(p, offset=offset) == int(first[-1])
    p, behind = row(V, first, 0)
    assert draw(p, offset=offset) == behind


@pytest.mark.parametrize("offset", [0, 1])
def test_sums_of_a_row_of_which_the_draft_leaves_nothing(offset):
    V = 1 << 22
    j = torch.arange(1 << 18)
    first = j[j % 2048 < 8]
    for below in (10, 0):
        p, behind = row(V, first, below)
        want = int(first[-1]) if below else behind
        assert draw(p, q=p, token=V - 1, offset=offset) == want
