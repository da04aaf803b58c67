"""Token log probabilities, entropies and top alternatives against the FP64
oracle.  Alternatives are exact: values are compared as they are, ties go to the
lowest token.

Bounds.  z is a sum of at most 33 terms one after the other in a thread for each
of its tiles, then pairwise: with exponentials good to 2^-21 (two units in the
last place, and half a unit of an argument of up to 100 that counts: beyond that a
term is below e^-100), relative error below 2^-21 + (33 tiles + 20) 2^-24, tiles
under 40 here: 2^-13.5 at worst and absolute in log z.  x - m is rounded once,
2^-24 of it, and so is the result.  The entropy's sum has the same relative error
on each of its terms, which are of one sign."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = 2.0 ** -13.5
i32 = torch.int32


def run(x, tokens, top, entropy=True, **kw):
    rows = len(tokens)
    lp = torch.full((rows,), 7.0, device="cuda")
    ent = torch.full((rows,), 7.0, device="cuda") if entropy else None
    tt = torch.full((rows, top), -7, dtype=i32, device="cuda") if top else None
    tl = torch.full((rows, top), 7.0, device="cuda") if top else None
    kda.kda_token_logprobs(x, torch.as_tensor(tokens, dtype=i32).cuda(), lp, entropy=ent, top_tokens=tt, top_logprobs=tl, **kw)
    return lp, ent, tt, tl


def close(got, want):
    """got against want, which may be past FP32's range."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        same = (got == want.astype(np.float32)) | (np.abs(got - want) <= REL + 2.0 ** -22 * np.abs(np.where(np.isfinite(want), want, 0)))
    return same.all()


def compare(x, tokens, top, got):
    lp, ent, tt, tl = (None if g is None else g.cpu().numpy() for g in got)
    x = x.float().cpu().numpy()
    for r, t in enumerate(tokens):
        if t == -1:
            assert lp[r] == 0 and (ent is None or ent[r] == 0) and (not top or ((tt[r] == -1).all() and (tl[r] == 0).all()))
            continue
        want = so.logprobs(x[r], t, top)
        assert close(lp[r], want[0]), (r, lp[r], want[0])
        if ent is not None:
            assert abs(ent[r] - want[1]) <= REL * (1 + abs(want[1])) and ent[r] >= -2.0 ** -20, (r, ent[r], want[1])
        if top:
            assert (tt[r] == want[2]).all(), (r, tt[r], want[2])
            assert close(tl[r], want[3]), (r, tl[r], want[3])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (2, 2, 5), (3, 7, 0), (2, 31, 32), (5, 1000, 5), (4, 8191, 20), (3, 8193, 32),
                                            (7, 50257, 20), (1, 32000, 1), (2, 131072, 5), (1, 151936, 8), (600, 513, 3),
                                            (500, 20001, 20), (1, 262149, 32)])
def test_rows(dtype, rows, vocab, top):
    gen = torch.Generator().manual_seed(rows * vocab)
    x = (torch.randn(rows, vocab, generator=gen) * 2.5).to(DT[dtype])
    tokens = torch.randint(0, vocab, (rows,), generator=gen).tolist()
    if rows > 2:
        tokens[1] = -1
    err = torch.zeros(1, dtype=i32, device="cuda")
    got = run(x.cuda(), tokens, top, err_flag=err)
    assert err.item() == 0
    some = range(rows) if rows < 20 else range(0, rows, 37)
    for r in some:
        compare(x[r:r + 1], tokens[r:r + 1], top, [None if g is None else g[r:r + 1] for g in got])
    again = run(x.cuda(), tokens, top)
    assert all(g is None or torch.equal(g, h) for g, h in zip(got, again))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("offset,pad", [(1, 0), (3, 5), (0, 1), (7, 2)])
def test_alignment_and_padding(dtype, offset, pad):
    """Rows that start anywhere, and apart by more than their length; what lies
    around them is not read as theirs."""
    rows, vocab = 5, 9001
    gen = torch.Generator().manual_seed(3)
    big = torch.full((offset + rows * (vocab + pad),), 1e4, dtype=DT[dtype])
    x = big[offset:].view(rows, vocab + pad)[:, :vocab]
    x.copy_(torch.randn(rows, vocab, generator=gen) * 3)
    tokens = [0, vocab - 1, 5, -1, 4000]
    dev = big.cuda()[offset:].view(rows, vocab + pad)[:, :vocab]
    assert dev.data_ptr() % 16 == (offset * big.element_size()) % 16
    compare(x, tokens, 6, run(dev, tokens, 6))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("vocab", [5, 300, 20000, 70000])
def test_special_rows(dtype, vocab):
    """Equal values, falling and rising ones, masks, infinities, NaN, rows with
    nothing left."""
    dt, top = DT[dtype], 20
    low = torch.finfo(dt).min
    i = torch.arange(vocab)
    x = torch.zeros(14, vocab)
    x[1] = -i / vocab * 100
    x[2] = i / vocab * 100
    x[3] = torch.where(i % 7 == 3, 1.0, -torch.inf)
    x[4] = -torch.inf
    x[5] = torch.where(i == vocab - 1, 2.0, -torch.inf)
    x[6] = torch.where(i < vocab // 2, float(low), float("nan"))
    x[7] = torch.where(i % 3 == 0, float("nan"), torch.randn(vocab, generator=torch.Generator().manual_seed(1)))
    x[8, vocab // 2] = torch.inf
    x[9] = torch.inf
    x[10] = float("nan")
    x[11] = torch.where(i % 2 == 0, -0.0, 0.0)
    x[12] = torch.where(i < 900, (i % 5).float(), -torch.inf)
    x[13] = low
    x = x.to(dt)
    tokens = [vocab - 1, 0, vocab - 1, 3, 1, vocab - 1, 0, 1, vocab // 2, 2, 0, 4, 4, 0]
    compare(x, tokens, top, run(x.cuda(), tokens, top))
    compare(x, tokens, 0, run(x.cuda(), tokens, 0, entropy=False))


def test_far_apart_values():
    """Shares too small for FP32, and logits next to its largest number."""
    x = torch.zeros(3, 10000)
    x[0] = -200.0
    x[0, 77] = 0.0
    x[1] = -3e38
    x[1, 5] = 3e38
    x[2] = 3.4e38
    tokens = [78, 6, 9999]
    compare(x, tokens, 3, run(x.cuda(), tokens, 3))


def test_bad_tokens_are_flagged():
    x = torch.randn(4, 100)
    err = torch.zeros(1, dtype=i32, device="cuda")
    got = run(x.cuda(), [3, 100, -2, 99], 4, err_flag=err)
    assert err.item() == kda.KDA_DEVERR_TOKEN
    compare(x, [3, -1, -1, 99], 4, got)


def test_rows_far_from_the_start():
    """Rows that begin past 2^32 elements."""
    big = torch.empty((1 << 32) + 5000, dtype=torch.bfloat16, device="cuda")
    stride = 1 << 31
    x = big.as_strided((3, 4999), (stride, 1))
    x.copy_(torch.randn(3, 4999))
    compare(x, [1, 2, 4998], 5, run(x, [1, 2, 4998], 5))


def test_captured_and_on_another_stream():
    x = torch.randn(6, 40000, device="cuda")
    tokens = torch.tensor([1, 2, 3, -1, 5, 39999], dtype=i32, device="cuda")
    out = [torch.zeros(6, device="cuda"), torch.zeros(6, device="cuda"), torch.zeros(6, 5, dtype=i32, device="cuda"),
           torch.zeros(6, 5, device="cuda")]
    call = lambda **kw: kda.kda_token_logprobs(x, tokens, out[0], out[1], out[2], out[3], **kw)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        x.normal_()
        graph.replay()
        compare(x, tokens.tolist(), 5, out)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    x.normal_()
    st.wait_stream(torch.cuda.current_stream())
    call(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    compare(x, tokens.tolist(), 5, out)


@pytest.mark.parametrize("vocab", [2, 9, 300, 5000])
@pytest.mark.parametrize("dtype", list(DT))
def test_all_but_certain_tokens(dtype, vocab):
    """Log probabilities and entropies near 0 are exact relative to themselves.  Logits
    are multiples of 1/8 between -16 and 26, so differences of them are exact; in units of
    2^-24: an exponential 4 and 42 (2^-22 of the approximation; half a unit of an argument
    of up to 61 in units of ln 2), 24 for the sums of 20 entries a thread with the joins,
    4 for the logarithm and the quotient: 74, below 2^-17."""
    gen = torch.Generator().manual_seed(vocab)
    rows = 12
    x = -torch.randint(0, 8 * 16, (rows, vocab), generator=gen).float() / 8
    at = torch.randint(0, vocab, (rows,), generator=gen)
    x[torch.arange(rows), at] = 4.0 + 2 * torch.arange(rows).clamp(max=14)
    got = run(x.to(DT[dtype]).cuda(), at, 1)
    lp = torch.log_softmax(x.double(), -1)
    r = torch.exp(x.double() - x.double().amax(-1, keepdim=True))
    r[torch.arange(rows), at] = 0
    want = -torch.log1p(r.sum(-1))
    entropy = -(lp * lp.exp()).masked_fill(torch.nn.functional.one_hot(at, vocab).bool(), 0).sum(-1) - want * want.exp()
    for name, g, w in (("logprobs", got[0], want), ("entropy", got[1], entropy), ("top_logprobs", got[3][:, 0], want)):
        off = ((g.double().cpu() - w).abs() / w.abs().clamp(min=1e-30)).max().item()
        assert off <= 2.0 ** -17, f"{name}: {off:.2e}"


@pytest.mark.parametrize("dtype", list(DT))
def test_candidates_late_in_long_rows(dtype):
    """Rows of many tiles, a CTA a row (504 rows), whose candidates come late, in crowds, in
    equal values or between entries without a probability."""
    vocab, top = 70000, 32  # (rows that start alike are summed alike)
    i = torch.arange(vocab)
    gen = torch.Generator().manual_seed(9)
    x = torch.zeros(8, vocab)
    x[0] = i / vocab * 50  # rising: all of it
    x[1] = torch.where(i < 40000, torch.randn(vocab, generator=gen), 5.0)  # equal ones behind 40000 others
    x[2] = torch.randn(vocab, generator=gen) + (i // 8192).float()  # each tile above the one before
    x[3] = torch.where(torch.rand(vocab, generator=gen) < 0.6, -torch.inf, torch.randn(vocab, generator=gen) * 4)
    x[4] = torch.where(i % 4096 < 600, 30.0 + (i // 30000).float(), 0.0)  # crowds of equal ones
    x[5] = torch.where(i > vocab - 20, 1.0, -torch.inf)  # fewer than asked for, at the end
    for r, n in ((6, 4), (7, 8)):  # crowds that 31 threads of 256 read
        x[r] = torch.where(i // n % 256 < 31, 10 + i / vocab, torch.rand(vocab, generator=gen))
    x = x.to(DT[dtype])
    tokens = [vocab - 1, 3, 65000, 7, 60000, vocab - 2, 9, 11]
    got = run(x.cuda().repeat(63, 1), tokens * 63, top)
    for g in got:
        assert torch.equal(g.view(63, 8, *g.shape[1:]), g[:8].expand(63, 8, *g.shape[1:]))
    compare(x, tokens, top, [g[:8] for g in got])
