"""Verification of drafted tokens against the FP64 oracle: whole numbers, equal
or wrong.  Random rows keep the draw away from borders between tokens by more
than the oracle's own rounding; the border tests use weights that are multiples
of 2^-12, whose sums are exact in any order."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu


def probs(rng, shape, dtype, spread=2.5):
    x = torch.softmax(torch.from_numpy(rng.normal(size=shape) * spread), -1)
    return x.to(dtype)


def f64(x):
    return x.double().numpy()


def out(*shape):
    return torch.full(shape, -7, dtype=torch.int32, device="cuda")


def pad_rows(x, stride, offset=0):
    """The same rows `stride` elements apart, starting `offset` elements into a buffer."""
    B, T, V = x.shape
    buf = torch.full((offset + B * T * stride,), float("nan"), dtype=x.dtype).cuda()
    view = buf[offset:].view(B, T, stride)[:, :, :V]
    view.copy_(x)
    return view


def chain(target, draft, tokens, u, lengths=None, err=None):
    B, T = tokens.shape
    acc, nxt = out(B), out(B)
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    kda.kda_accept_chain(dev(target), dev(draft), dev(tokens), dev(u), acc, nxt, lengths=dev(lengths), err_flag=err)
    return acc.cpu().tolist(), nxt.cpu().tolist()


def tree(target, tokens, parent, u, lengths=None, err=None):
    B, T = tokens.shape
    acc, path, nxt = out(B), out(B, T), out(B)
    kda.kda_accept_tree(target.cuda(), tokens.cuda(), parent.cuda(), u.cuda(), acc, path, nxt,
                        lengths=None if lengths is None else lengths.cuda(), err_flag=err)
    return acc.cpu().tolist(), path.cpu().tolist(), nxt.cpu().tolist()


@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (3, 2, 2), (5, 6, 7), (2, 6, 1000), (7, 8, 4097), (48, 6, 32000),
                                   (1, 6, 131072), (3, 4, 50257), (300, 3, 129)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("with_draft", [True, False])
def test_chain(B, T, V, dtype, with_draft):
    rng = np.random.default_rng(B * 1000 + V)
    target = probs(rng, (B, T, V), dtype)
    draft = probs(rng, (B, max(T - 1, 1), V), dtype) if with_draft else None
    if with_draft and T > 1:  # a draft model near the target
        draft = (0.7 * target[:, :T - 1].float() + 0.3 * draft.float()).to(dtype)
    tokens = torch.from_numpy(rng.integers(0, V, (B, T))).int()
    for i in range(1, T):
        src = (draft[:, i - 1] if with_draft else target[:, i - 1]).float()
        tokens[:, i] = torch.multinomial(src, 1).view(-1).int()
    u = torch.from_numpy(rng.random((B, T)).astype(np.float32))
    lengths = torch.from_numpy(rng.integers(0, T + 1, B)).int() if B > 2 else None
    acc, nxt = chain(target, draft, tokens, u, lengths)
    for r in range(B):
        n = T if lengths is None else int(lengths[r])
        want = so.accept_chain(f64(target[r]), None if draft is None else f64(draft[r]), tokens[r].tolist(),
                               u[r].numpy(), n)
        assert (acc[r], nxt[r]) == want, (r, n)


@pytest.mark.parametrize("B,T,V", [(1, 1, 3), (4, 2, 2), (9, 16, 30), (16, 6, 50257), (2, 40, 1000), (3, 1024, 17)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tree(B, T, V, dtype):
    rng = np.random.default_rng(T * 100 + V)
    target = probs(rng, (B, T, V), dtype, spread=1.5)
    parent = torch.tensor([[-1] + [int(rng.integers(0, i)) for i in range(1, T)] for _ in range(B)]).int()
    tokens = torch.from_numpy(rng.integers(0, V, (B, T))).int()
    for r in range(B):
        for i in range(1, T):  # likely tokens, some of them tried twice
            top = target[r, parent[r, i]].float().topk(min(4, V)).indices
            tokens[r, i] = top[int(rng.integers(0, len(top)))]
    u = torch.from_numpy(rng.random((B, T)).astype(np.float32))
    lengths = torch.from_numpy(rng.integers(0, T + 1, B)).int() if B > 2 else None
    acc, path, nxt = tree(target, tokens, parent, u, lengths)
    for r in range(B):
        n = T if lengths is None else int(lengths[r])
        a, p, x = so.accept_tree(f64(target[r]), tokens[r].tolist(), parent[r].tolist(), u[r].numpy(), n)
        assert (acc[r], nxt[r]) == (a, x), (r, n)
        assert path[r] == p + [-1] * (T - len(p))


@pytest.mark.parametrize("V,at", [(64, 0), (64, 40), (4096, 4095), (20000, 12345), (100000, 99999)])
def test_draw_on_a_border_takes_the_next_token(V, at):
    """Whole weight 1 in steps of 2^-12; u exactly the sum up to token `at`:
    that sum does not exceed it, so the next token with weight is drawn."""
    p = torch.zeros(1, 1, V)
    hot = torch.linspace(0, V - 1, 32).round().long().unique()
    hot = torch.cat([hot, torch.tensor([at])]).unique()
    steps = torch.full((len(hot),), 4096 // len(hot))
    steps[0] += 4096 - steps.sum()
    p[0, 0, hot] = steps / 4096.0
    cum = p[0, 0].double().cumsum(0)
    tokens = torch.zeros(1, 1).int()
    for u, want in ((float(cum[at]), int(hot[hot > at][0]) if (hot > at).any() else at),
                    (float(cum[at]) - 2.0 ** -13, at), (0.0, int(hot[0]))):
        if u >= 1:
            u, want = 1 - 2.0 ** -24, int(hot[-1])
        assert chain(p, None, tokens, torch.tensor([[u]]))[1] == [want]


def test_odd_values_and_empty_rows():
    """NaN, negative and infinite entries have no weight; where max(p - q, 0)
    leaves nothing the draw is from p; a row with nothing at all gives -1."""
    V = 70
    p = torch.zeros(4, 2, V)
    p[:, :, 5], p[:, :, 60] = 0.25, 0.75
    p[:, :, 1], p[:, :, 2], p[:, :, 3] = float("nan"), float("inf"), -1.0
    q = p[:, :1].clone()
    p[2], q[3] = 0.0, 0.0
    tokens = torch.tensor([[0, 1], [0, 2], [0, 5], [0, 5]]).int()
    u = torch.tensor([[0.3, 0.0], [0.1, 0.0], [0.5, 0.0], [0.2, 0.5]])
    acc, nxt = chain(p, q, tokens, u)
    # 0, 1: the draft has no weight and falls, p - q leaves nothing; 2: nothing at all; 3: q = 0 stands
    assert acc == [0, 0, 0, 1] and nxt == [60, 5, -1, 5]
    # a tree whose tried tokens took all of the row
    p = torch.zeros(1, 3, V)
    p[0, 0, 7], p[0, 0, 8] = 0.5, 0.5
    acc, path, nxt = tree(p, torch.tensor([[0, 7, 8]]).int(), torch.tensor([[-1, 0, 0]]).int(),
                          torch.tensor([[0.75, 1.0, 1.0]]))
    assert (acc, path, nxt) == ([0], [[0, -1, -1]], [8])


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("stride", [1024, 1001, 1027])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_alignments(offset, stride, dtype):
    rng = np.random.default_rng(stride + offset)
    B, T, V = 3, 4, 1001
    target, draft = probs(rng, (B, T, V), dtype), probs(rng, (B, T - 1, V), dtype)
    tokens = torch.from_numpy(rng.integers(0, V, (B, T))).int()
    u = torch.from_numpy(rng.random((B, T)).astype(np.float32))
    plain = chain(target, draft, tokens, u)
    assert plain == chain(pad_rows(target, stride, offset), pad_rows(draft, stride + 5, offset), tokens, u)
    want = [so.accept_chain(f64(target[r]), f64(draft[r]), tokens[r].tolist(), u[r].numpy(), T) for r in range(B)]
    assert list(zip(*plain)) == want


def test_device_errors():
    rng = np.random.default_rng(0)
    target = probs(rng, (3, 3, 20), torch.float32)
    u = torch.full((3, 3), 0.01)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens = torch.tensor([[0, 20, 1], [0, -1, 1], [0, int(target[2, 0].argmax()), int(target[2, 1].argmax())]]).int()
    acc, nxt = chain(target, None, tokens, u, err=err)
    assert int(err) == kda.KDA_DEVERR_TOKEN and acc == [0, 0, 2] and all(0 <= x < 20 for x in nxt)
    err.zero_()
    acc, nxt = chain(target, None, tokens.clamp(0, 19), u, lengths=torch.tensor([4, -1, 0]).int(), err=err)
    assert int(err) == kda.KDA_DEVERR_SEQLENS and acc == nxt == [-1, -1, -1]
    err.zero_()
    parent = torch.tensor([[-1, 1, 0], [0, 0, 1], [-1, 0, 1]]).int()
    acc, path, nxt = tree(target, tokens.clamp(0, 19), parent, u, err=err)
    assert int(err) == kda.KDA_DEVERR_PARENT and acc[:2] == nxt[:2] == [-1, -1]
    assert path[:2] == [[-1] * 3] * 2 and path[2][0] == 0


def test_in_a_graph_with_new_numbers():
    rng = np.random.default_rng(1)
    B, T, V = 4, 5, 3000
    target, draft = probs(rng, (B, T, V), torch.float32).cuda(), probs(rng, (B, T - 1, V), torch.float32).cuda()
    tokens = torch.from_numpy(rng.integers(0, V, (B, T))).int().cuda()
    u, acc, nxt = torch.zeros(B, T, device="cuda"), out(B), out(B)
    kda.kda_accept_chain(target, draft, tokens, u, acc, nxt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_accept_chain(target, draft, tokens, u, acc, nxt)
    for _ in range(3):
        u.copy_(torch.from_numpy(rng.random((B, T)).astype(np.float32)))
        graph.replay()
        want = chain(target, draft, tokens, u)
        assert (acc.cpu().tolist(), nxt.cpu().tolist()) == want
