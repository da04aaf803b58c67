"""The gated delta rule with one decay per value head against the FP64 oracle:
prefill, decode, chain and tree verify.

Tolerances.  Outputs: the framework's 2e-2 RMS on top of the 16-bit output's
own rounding (assert_o_close).  States behind T single tokens: every token
rounds an element some 60 times in FP32 at most (16 products and sums a lane,
3 shuffle sums, norms, gate, update), 60 2^-24 < 2^-18 of the largest value.
Prefill states: each of the four operands that a chunk splits in two 16-bit
halves keeps 2^-16 of its value, 2^-14 together; a state's largest elements are
about 4 times its RMS, so 2^-12 RMS."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so
from tests.gpu_util import assert_o_close, host_f64, rms

pytestmark = pytest.mark.gpu
K = 128
SCALE = K ** -0.5


def make(seed, tokens, H, HV, slots, f16=False, given=False, gb_rows=None, raw_beta=True, l2=True):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float16 if f16 else torch.bfloat16
    size = 1.0 if l2 else K ** -0.5
    d = dict(q=torch.randn(tokens, H, K, generator=g) * size, k=torch.randn(tokens, H, K, generator=g) * size,
             v=torch.randn(tokens, HV, K, generator=g))
    d = {n: x.to(dt) for n, x in d.items()}
    gb = gb_rows or tokens
    d["A_log"] = torch.empty(HV).uniform_(0, 2.7, generator=g)
    d["dt_bias"] = torch.empty(HV).uniform_(-6, -2, generator=g)
    a = torch.randn(gb, HV, generator=g)
    b = torch.randn(gb, HV, generator=g)
    if not raw_beta:
        b = torch.rand(gb, HV, generator=g)
    if given:
        a = -torch.exp(torch.empty(gb, HV).uniform_(-9, 2, generator=g))
        d["A_log"] = d["dt_bias"] = None
    else:
        a = a.to(dt)
    a[tokens:], b[tokens:] = float("nan"), float("nan")
    d["a"], d["b"] = a, b.to(dt)
    d["pool"] = torch.randn(slots, HV, K, K, generator=g) * 0.02
    d["idx"] = torch.randperm(slots, generator=g).int()
    d["dims"] = kda.dims(H, HV=HV, dtype=kda.KDA_DTYPE_F16 if f16 else kda.KDA_DTYPE_BF16)
    d["l2"], d["raw_beta"], d["dt"] = l2, raw_beta, dt
    return d


def gate_of(d):
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    return kda.ScalarGate(A_log=dev(d["A_log"]), dt_bias=dev(d["dt_bias"]), beta_is_raw=d["raw_beta"],
                          use_qk_l2norm=d["l2"])


def f64(x):
    return x.double().numpy()


def oracle_rows(d, rows, S, parents=None):
    al, be = so.gdn_gate(f64(d["a"][rows]), f64(d["b"][rows]), None if d["A_log"] is None else f64(d["A_log"]),
                         None if d["dt_bias"] is None else f64(d["dt_bias"]), d["raw_beta"])
    return so.gdn_sequence(S, f64(d["q"][rows]), f64(d["k"][rows]), f64(d["v"][rows]), al, be, SCALE, d["l2"],
                           parents)


def assert_state(got, ref, tol):
    got = host_f64(got) if isinstance(got, torch.Tensor) else got
    assert np.isfinite(got).all()
    err = np.abs(got - ref).max() if ref.size else 0.0
    assert err <= tol, (err, tol)


def prefill(d, lengths, idx=None, err=None, intermediate=None, pool=None, stream=None, fixed=False):
    T = sum(lengths)
    cu = torch.tensor(np.cumsum([0] + list(lengths)), dtype=torch.int32).cuda()
    idx = d["idx"][:len(lengths)] if idx is None else idx
    pool = d["pool"].cuda() if pool is None else pool
    o = torch.full((T, d["dims"].HV, K), 7.0, dtype=d["dt"], device="cuda")
    kda.kda_gdn_prefill(d["dims"], gate_of(d), d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), d["a"].cuda(),
                        d["b"].cuda(), pool, idx.cuda(), None if fixed else cu, len(lengths), o,
                        intermediate=intermediate, err_flag=err, stream=stream)
    return o, pool


def check_prefill(d, lengths, o, pool, idx=None, intermediate=None):
    idx = (d["idx"] if idx is None else idx).tolist()
    ref_pool = f64(d["pool"]).copy()
    t0 = chunk = 0
    outs, firsts = [], []
    for n, L in enumerate(lengths):
        S0 = ref_pool[idx[n]].copy()
        out, states = oracle_rows(d, slice(t0, t0 + L), S0)
        if L:
            outs.append(out)
            ref_pool[idx[n]] = states[-1]
            firsts += [S0 if c == 0 else states[c * 64 - 1] for c in range(-(-L // 64))]
        t0 += L
        chunk += -(-L // 64)
    if outs:
        assert_o_close(o, np.concatenate(outs))
    tol = 2.0 ** -12 * rms(np.stack([ref_pool[idx[n]] for n in range(len(lengths))]))
    assert_state(pool, ref_pool, tol)
    rest = [s for s in range(len(ref_pool)) if s not in idx[:len(lengths)]]
    assert torch.equal(pool[rest].cpu(), d["pool"][rest])
    if intermediate is not None:
        assert_state(intermediate[:chunk], np.stack(firsts), tol)


@pytest.mark.parametrize("lengths", [[1], [2], [63], [64], [65], [127, 1, 0, 200], [0, 5], [130, 64, 64, 17, 1, 1]])
@pytest.mark.parametrize("f16", [False, True])
def test_prefill_lengths(lengths, f16):
    d = make(1, sum(lengths), 2, 2, len(lengths) + 2, f16=f16, gb_rows=sum(lengths) + 9)
    o, pool = prefill(d, lengths)
    check_prefill(d, lengths, o, pool)


@pytest.mark.parametrize("H,HV,given,raw_beta,l2", [(1, 1, True, True, True), (2, 8, False, True, True),
                                                   (4, 4, True, False, True), (1, 3, False, True, False),
                                                   (16, 16, False, False, True), (8, 32, True, True, True)])
def test_prefill_heads_and_folds(H, HV, given, raw_beta, l2):
    lengths = [97, 33, 150]
    d = make(2, sum(lengths), H, HV, 5, given=given, raw_beta=raw_beta, l2=l2)
    o, pool = prefill(d, lengths)
    check_prefill(d, lengths, o, pool)


@pytest.mark.parametrize("f16", [False, True])
def test_prefill_long_and_slow_decay(f16):
    """The state carries over 32 chunks with next to no decay."""
    lengths = [2048]
    d = make(3, 2048, 2, 2, 2, f16=f16, given=True)
    d["a"] = -torch.rand(2048, 2) * 1e-3
    inter = torch.full((32, 2, K, K), 9.0, device="cuda")
    o, pool = prefill(d, lengths, intermediate=inter)
    check_prefill(d, lengths, o, pool, intermediate=inter)


def test_prefill_chunk_states_and_their_capacity():
    lengths = [70, 0, 64, 129, 3]
    d = make(4, sum(lengths), 2, 4, 7)
    inter = torch.full((7, 4, K, K), 9.0, device="cuda")
    o, pool = prefill(d, lengths, intermediate=inter)
    check_prefill(d, lengths, o, pool, intermediate=inter)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    short = torch.full((7, 4, K, K), 9.0, device="cuda")
    prefill(d, lengths, intermediate=short[:4], err=err)
    assert int(err) == kda.KDA_DEVERR_INTERMEDIATE
    assert torch.equal(short[:4], inter[:4]) and bool((short[4:] == 9).all())


def test_prefill_decay_extremes():
    """Log-decays of zero, of -inf (the state is dropped) and far below FP32's
    range beside slow ones: factors stay finite, slow ones keep their precision."""
    d = make(5, 200, 1, 2, 2, given=True)
    d["a"][:] = -1e-4
    d["a"][::7] = 0.0
    d["a"][20, 0] = -float("inf")
    d["a"][100:103] = -1e30
    d["a"][150] = -40.0
    o, pool = prefill(d, [200])
    d["a"] = d["a"].clamp(min=-700)  # exp(-700) is 0 beside everything here, and finite in the oracle
    check_prefill(d, [200], o, pool)


def test_prefill_other_sequences_do_not_leak():
    """NaN and infinities in the rows of one sequence reach neither its
    neighbours in the same 64-row tile nor the next one's state."""
    lengths = [70, 40, 30]
    d = make(6, 140, 1, 1, 4)
    clean = {n: d[n].clone() for n in ("q", "k", "v")}
    for n, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan"))):
        d[n][70:110] = bad
    o, pool = prefill(d, lengths)
    d.update(clean)
    ref, ref_pool = prefill(d, lengths)
    keep = list(range(70)) + list(range(110, 140))
    assert torch.equal(o[keep], ref[keep])
    for n in (0, 2):
        s = int(d["idx"][n])
        assert torch.equal(pool[s], ref_pool[s])


def test_prefill_carried_over_calls_equals_one_call():
    d = make(7, 256, 2, 2, 2)
    whole, pool = prefill(d, [256])
    part = dict(d)
    p = d["pool"].cuda()
    got = []
    for t0, t1 in ((0, 128), (128, 256)):
        part.update({n: d[n][t0:t1] for n in ("q", "k", "v", "a", "b")})
        o, _ = prefill(part, [t1 - t0], pool=p)
        got.append(o)
    assert torch.equal(torch.cat(got), whole) and torch.equal(p, pool)


def test_prefill_padding_bad_slot_and_bad_bounds():
    d = make(8, 90, 1, 2, 4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor([2, -1, 9], dtype=torch.int32)
    o, pool = prefill(d, [30, 30, 30], idx=idx, err=err)
    assert int(err) == kda.KDA_DEVERR_SLOT
    assert bool((o[30:] == 0).all()) and bool((o[:30] != 0).any())
    assert torch.equal(pool[[0, 1, 3]].cpu(), d["pool"][[0, 1, 3]])
    # bounds that go back, or do not end at the last token: flagged, nothing out of range
    for cu in ([0, 60, 30, 90], [0, 30, 60, 80], [3, 30, 60, 90]):
        err.zero_()
        o = torch.zeros(90, 2, K, dtype=d["dt"], device="cuda")
        kda.kda_gdn_prefill(d["dims"], gate_of(d), d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), d["a"].cuda(),
                            d["b"].cuda(), d["pool"].cuda(), torch.tensor([0, 1, 2], dtype=torch.int32).cuda(),
                            torch.tensor(cu, dtype=torch.int32).cuda(), 3, o, err_flag=err)
        assert int(err) == kda.KDA_DEVERR_SEQLENS


def test_prefill_fixed_layout_many_sequences_and_streams():
    d = make(9, 20 * 40, 2, 2, 50)
    o, pool = prefill(d, [40] * 20)
    check_prefill(d, [40] * 20, o, pool)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, pool2 = prefill(d, [40] * 20, fixed=True)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(pool, pool2)


@pytest.mark.parametrize("f16", [False, True])
def test_prefill_many_sequences(f16):
    """Enough (sequence, head) pairs for the wide state kernel, with ragged,
    empty and padding sequences, grouped heads and chunk-start states."""
    rng = np.random.default_rng(0)
    lengths = [int(x) for x in rng.integers(0, 150, 70)]
    lengths[3], lengths[5], lengths[7] = 400, 64, 1
    d = make(14, sum(lengths), 2, 4, 75, f16=f16, given=True, gb_rows=sum(lengths) + 3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    inter = torch.full((sum(-(-L // 64) for L in lengths), 4, K, K), 9.0, device="cuda")
    o, pool = prefill(d, lengths, err=err, intermediate=inter)
    assert int(err) == 0
    check_prefill(d, lengths, o, pool, intermediate=inter)
    idx = d["idx"][:70].clone()
    idx[4] = -1
    o2, pool2 = prefill(d, lengths, idx=idx)
    t0 = sum(lengths[:4])
    keep = [t for t in range(sum(lengths)) if not t0 <= t < t0 + lengths[4]]
    assert torch.equal(o2[keep], o[keep]) and bool((o2[t0:t0 + lengths[4]] == 0).all())
    s = int(d["idx"][4])
    assert torch.equal(pool2[s].cpu(), d["pool"][s])


@pytest.mark.parametrize("lengths,H,HV", [
    ([300], 2, 8),                            # 8 value columns a CTA
    ([300], 4, 16),                           # 16
    ([190, 70], 8, 16),                       # 32
    ([1500, 30, 64, 65, 0, 129, 1], 8, 16),   # one sequence by columns, the others whole heads
    ([300, 1400, 90, 1301, 7, 200], 1, 8),    # two
    ([130] * 12, 4, 16),                      # none
    ([100, 33], 4, 64),                       # no sequence fits by columns
    ([int(x) for x in np.random.default_rng(3).integers(0, 70, 140)], 1, 2),  # too many to rank
])
@pytest.mark.parametrize("f16", [False, True])
def test_prefill_forms_of_the_state_pass(lengths, H, HV, f16):
    d = make(16, sum(lengths), H, HV, len(lengths) + 1, f16=f16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    inter = torch.full((sum(-(-L // 64) for L in lengths), HV, K, K), 9.0, device="cuda")
    o, pool = prefill(d, lengths, err=err, intermediate=inter)
    assert int(err) == 0
    check_prefill(d, lengths, o, pool, intermediate=inter)


def test_prefill_and_decode_in_a_graph():
    d = make(10, 130, 2, 4, 3)
    x = {n: d[n].cuda() for n in ("q", "k", "v", "a", "b", "idx")}
    gate = gate_of(d)
    cu = torch.tensor([0, 100, 130], dtype=torch.int32).cuda()
    eager, pool = prefill(d, [100, 30])
    packed = torch.randn(2, (2 * 2 + 4) * K, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    od = torch.zeros(2, 4, K, dtype=d["dt"], device="cuda")

    def both(o, p):
        kda.kda_gdn_prefill(d["dims"], gate, x["q"], x["k"], x["v"], x["a"], x["b"], p, x["idx"], cu, 2, o)
        kda.kda_gdn_decode_packed(d["dims"], gate, packed, x["a"][:2], x["b"][:2], p, x["idx"], od)

    p0, o0 = d["pool"].cuda(), torch.zeros_like(eager)
    both(o0, p0)
    want = od.clone()
    p, o = d["pool"].cuda(), torch.zeros_like(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(o, p)
    p.copy_(d["pool"])
    od.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, eager) and torch.equal(p, p0) and torch.equal(od, want)


def packed_of(d, rows):
    return torch.cat([d[n].reshape(rows, -1) for n in ("q", "k", "v")], 1)


@pytest.mark.parametrize("B,H,HV,f16,given", [(1, 1, 1, False, False), (3, 2, 4, True, False), (17, 4, 4, False, True),
                                             (48, 16, 32, False, False), (2, 16, 16, True, True)])
def test_decode(B, H, HV, f16, given):
    d = make(11, B, H, HV, B + 3, f16=f16, given=given)
    idx = d["idx"][:B].clone()
    if B > 2:
        idx[1] = -1
    wide = torch.zeros(B, (2 * H + HV) * K + 24, dtype=d["dt"])  # rows further apart than they are long
    wide[:, :-24] = packed_of(d, B)
    pool, o = d["pool"].cuda(), torch.full((B, HV, K), 3.0, dtype=d["dt"], device="cuda")
    kda.kda_gdn_decode_packed(d["dims"], gate_of(d), wide.cuda(), d["a"].cuda(), d["b"].cuda(), pool, idx.cuda(), o)
    ref_pool, ref_o = f64(d["pool"]).copy(), np.zeros((B, HV, K))
    for r in range(B):
        if idx[r] >= 0:
            out, st = oracle_rows(d, slice(r, r + 1), ref_pool[idx[r]])
            ref_o[r], ref_pool[idx[r]] = out[0], st[0]
    assert_o_close(o, ref_o)
    assert_state(pool, ref_pool, 2.0 ** -18 * np.abs(ref_pool).max())
    rest = [s for s in range(B + 3) if s not in idx.tolist()]
    assert torch.equal(pool[rest].cpu(), d["pool"][rest])


@pytest.mark.parametrize("B,T,H,HV,tree,f16", [(1, 1, 1, 1, False, False), (2, 6, 2, 4, False, True), (5, 11, 1, 2, True, False),
                                              (16, 6, 4, 4, True, True), (16, 6, 16, 16, False, False)])
def test_verify_and_commit(B, T, H, HV, tree, f16):
    d = make(12, B * T, H, HV, B + 2, f16=f16)
    rng = np.random.default_rng(0)
    parents = np.array([[int(rng.integers(-1, i)) for i in range(T)] for _ in range(B)], np.int32)
    if not tree:
        parents[:] = np.arange(T) - 1
    pool = d["pool"].cuda()
    o = torch.zeros(B, T, HV, K, dtype=d["dt"], device="cuda")
    snap = torch.zeros(B, T, HV, K, K, device="cuda")
    args = (d["dims"], gate_of(d), packed_of(d, B * T).cuda(), d["a"].cuda(), d["b"].cuda(), B, T)
    idx = d["idx"][:B].cuda()
    if tree:
        kda.kda_gdn_verify_tree(*args, torch.from_numpy(parents).cuda(), pool, idx, o, snap)
    else:
        kda.kda_gdn_verify_chain(*args, pool, idx, o, snap)
    assert torch.equal(pool.cpu(), d["pool"])
    for r in range(B):
        out, st = oracle_rows(d, slice(r * T, (r + 1) * T), f64(d["pool"][d["idx"][r]]), parents[r])
        assert_o_close(o[r], out)
        assert_state(snap[r], st, 2.0 ** -18 * (T + 1) * np.abs(st).max())
    acc = torch.arange(B, dtype=torch.int32) % (T + 1) - 1
    kda.kda_commit(d["dims"], snap, B, T, acc.cuda(), pool, idx)
    for r in range(B):
        want = d["pool"][d["idx"][r]] if acc[r] < 0 else snap[r, int(acc[r])].cpu()
        assert torch.equal(pool[int(d["idx"][r])].cpu(), want)


def test_verify_refuses_on_the_device():
    d = make(13, 8, 1, 2, 4)
    pool = d["pool"].cuda()
    o = torch.full((2, 4, 2, K), 5.0, dtype=d["dt"], device="cuda")
    snap = torch.full((2, 4, 2, K, K), 5.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (d["dims"], gate_of(d), packed_of(d, 8).cuda(), d["a"].cuda(), d["b"].cuda(), 2, 4)
    par = torch.tensor([[-1, 0, 2, 1], [-1, 0, 0, 2]], dtype=torch.int32).cuda()  # node 2 its own parent
    kda.kda_gdn_verify_tree(*args, par, pool, torch.tensor([0, 1], dtype=torch.int32).cuda(), o, snap, err_flag=err)
    assert int(err) == kda.KDA_DEVERR_PARENT
    assert bool((o[0] == 0).all()) and bool((snap[0] == 5).all()) and bool((o[1] != 0).any())
    err.zero_()
    kda.kda_gdn_verify_chain(*args, pool, torch.tensor([4, -1], dtype=torch.int32).cuda(), o, snap, err_flag=err)
    assert int(err) == kda.KDA_DEVERR_SLOT and bool((o == 0).all())
