"""NaN, infinite and negative entries in rows that are read 16 bytes at a time, in
blocks of one size and of the other, and rows of more than 2^20 entries: against
the FP64 oracle."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu
ODD = (float("nan"), float("inf"), -float("inf"), -1.0, -0.0)


def f64(x):
    return x.double().numpy()


def out(*shape):
    return torch.full(shape, -7, dtype=torch.int32, device="cuda")


def spoilt(rng, shape, dtype, like=None):
    """Probabilities with odd entries; with `like`, a draft's, some of them at the
    target's own odd entries."""
    p = torch.softmax(torch.from_numpy(rng.normal(size=shape) * 2), -1)
    if like is not None:
        p = 0.5 * p + 0.5 * like.double().nan_to_num(0, 0, 0).clamp(min=0)
    p = p.to(dtype)
    V = shape[-1]
    for row in p.view(-1, V):
        at = rng.integers(0, V, min(V, 12))
        for k, j in enumerate(at):
            row[j] = ODD[k % len(ODD)]
    if like is not None:
        p = torch.where(torch.from_numpy(rng.random(shape) < 0.5) & ~like.isfinite(), like, p)
    return p


@pytest.mark.parametrize("V", [8, 72, 1000, 4096, 70000, 131072])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("with_draft", [True, False])
def test_chain_of_odd_rows(V, dtype, with_draft):
    rng = np.random.default_rng(V)
    B, T = 12, 4
    target = spoilt(rng, (B, T, V), dtype)
    draft = spoilt(rng, (B, T - 1, V), dtype, target[:, :T - 1]) if with_draft else None
    tokens = torch.from_numpy(rng.integers(0, V, (B, T))).int()
    for r in range(0, B, 2):  # odd entries as drafted tokens, and likely ones
        for i in range(1, T):
            row = target[r, i - 1].float()
            odd = (~(row > 0) | ~row.isfinite()).nonzero().view(-1)
            tokens[r, i] = int(odd[int(rng.integers(len(odd)))]) if i > 1 else int(row.nan_to_num(0, 0, 0).argmax())
    u = torch.from_numpy(rng.random((B, T)).astype(np.float32))
    u[::2, 1] = 0.0
    acc, nxt = out(B), out(B)
    kda.kda_accept_chain(target.cuda(), None if draft is None else draft.cuda(), tokens.cuda(), u.cuda(), acc, nxt)
    for r in range(B):
        want = so.accept_chain(f64(target[r]), None if draft is None else f64(draft[r]), tokens[r].tolist(), u[r].numpy(), T)
        assert (int(acc[r]), int(nxt[r])) == want, r


@pytest.mark.parametrize("V", [8, 72, 4096, 70000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_tree_of_odd_rows(V, dtype):
    rng = np.random.default_rng(V + 1)
    B, T = 9, 12
    target = spoilt(rng, (B, T, V), dtype)
    parent = torch.tensor([[-1] + [int(rng.integers(0, min(i, 3))) for i in range(1, T)] for _ in range(B)]).int()
    tokens = torch.from_numpy(rng.integers(0, V, (B, T))).int()
    u = torch.from_numpy(rng.random((B, T)).astype(np.float32))
    acc, path, nxt = out(B), out(B, T), out(B)
    kda.kda_accept_tree(target.cuda(), tokens.cuda(), parent.cuda(), u.cuda(), acc, path, nxt)
    for r in range(B):
        a, p, x = so.accept_tree(f64(target[r]), tokens[r].tolist(), parent[r].tolist(), u[r].numpy(), T)
        assert (int(acc[r]), int(nxt[r])) == (a, x), r
        assert path[r].tolist() == p + [-1] * (T - len(p))


@pytest.mark.parametrize("V", [(1 << 20) + 8, 1500000, 1500001, 5000000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_past_a_million(V, dtype):
    rng = np.random.default_rng(V)
    target = torch.softmax(torch.from_numpy(rng.normal(size=(1, 2, V)) * 3), -1).to(dtype)
    draft = torch.softmax(torch.from_numpy(rng.normal(size=(1, 1, V)) * 3), -1).to(dtype)
    d_target, d_draft = target.cuda(), draft.cuda()
    for k in range(6):
        tokens = torch.tensor([[0, int(rng.integers(V))]]).int()
        u = torch.from_numpy(rng.random((1, 2)).astype(np.float32))
        for q, dq in ((draft, d_draft), (None, None)):
            acc, nxt = out(1), out(1)
            kda.kda_accept_chain(d_target, dq, tokens.cuda(), u.cuda(), acc, nxt)
            assert (int(acc), int(nxt)) == so.accept_chain(f64(target[0]), None if q is None else f64(q[0]), tokens[0].tolist(),
                                                           u[0].numpy(), 2)
