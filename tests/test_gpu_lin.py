"""Linear attention with one decay per value head against the FP64 oracle:
prefill, packed decode, chain and tree verify."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so
from tests import lin_util as lu

pytestmark = pytest.mark.gpu
K = V = 128
SCALE = K ** -0.5
i32 = torch.int32


def case(lengths, H=1, HV=None, dtype="bf16", gate="raw", norm=True):
    return dict(lengths=lengths, H=H, HV=HV or H, dtype=dtype, gate=gate, norm=norm)


PREFILL = [
    case([1]), case([2], dtype="f16"), case([63, 64, 65], H=2), case([0, 1, 128, 129, 0], H=2, HV=4, dtype="f16"),
    case([200], gate="given"), case([333, 77], H=1, HV=4, gate="fixed", norm=False), case([130], gate="strong", dtype="f16"),
    case([257, 3], gate="out", H=2), case([190], gate="none", norm=False), case([190], gate="none", dtype="f16"),
    case([100, 90], gate="nobias", H=2, HV=2, dtype="f16", norm=False), case([1000, 64, 5, 700], H=1, HV=2, gate="fixed"),
    case([2100], H=1, HV=2, gate="fixed"), case([1537, 2, 640], H=2, gate="given", dtype="f16"),
]


def draw(c, seed, pad=7, spare=3):
    gen = torch.Generator().manual_seed(seed)
    T, n, dt = sum(c["lengths"]), len(c["lengths"]), lu.DT[c["dtype"]]
    x = dict(q=torch.randn(T, c["H"], K, generator=gen).to(dt), k=torch.randn(T, c["H"], K, generator=gen).to(dt),
             v=torch.randn(T, c["HV"], V, generator=gen).to(dt))
    x["A_log"], x["dt_bias"], x["a"] = lu.gate_inputs(gen, c["gate"], T + pad, c["HV"], dt)
    if x["a"] is not None:
        x["a"][T:] = float("nan")
    x["pool"] = torch.randn(n + spare, c["HV"], V, K, generator=gen) * 0.3
    x["idx"] = torch.randperm(n + spare, generator=gen)[:n].int()
    x["cu"] = torch.tensor([0] + np.cumsum(c["lengths"]).tolist(), dtype=i32)
    return x


def run(c, x, **kw):
    """A prefill of x: (o, pool), on the GPU."""
    up = {k: v.cuda() if v is not None else None for k, v in x.items()}
    o = torch.full((len(x["q"]), c["HV"], V), 7.0, dtype=lu.DT[c["dtype"]], device="cuda")
    kda.kda_lin_prefill(lu.dims(c), lu.scalar_gate(x["A_log"], x["dt_bias"], c["norm"]), up["q"], up["k"], up["v"], up["a"],
                        up["pool"], up["idx"], up["cu"], len(c["lengths"]), o, **kw)
    return o, up["pool"]


def compare(c, x, o, pool, parts=(0,), others=True):
    g = so.lin_decay(len(x["q"]), lu.host(x["a"]), lu.host(x["A_log"]), lu.host(x["dt_bias"]))
    want = lu.host(x["pool"])
    for n, slot in enumerate(x["idx"].tolist()):
        s = slice(int(x["cu"][n]), int(x["cu"][n + 1]))
        if s.start == s.stop:
            continue
        q, k, v = (lu.host(x[name][s]) for name in "qkv")
        o_ref, states = so.lin_sequence(want[slot], q, k, v, g[s], SCALE, c["norm"])
        o_b, s_b = lu.bounds(want[slot], q, k, v, g[s], SCALE, c["norm"], c["dtype"], parts=parts)
        lu.check(f"o of sequence {n}", o[s], o_ref, o_b, c["dtype"])
        lu.check(f"state of sequence {n}", pool[slot], states[-1], s_b)
    if not others:
        return
    rest = [s for s in range(len(want)) if s not in [i for i, L in zip(x["idx"].tolist(), c["lengths"]) if L]]
    assert torch.equal(pool[rest].cpu(), x["pool"][rest]), "a slot of no sequence"


@pytest.mark.parametrize("i", range(len(PREFILL)))
def test_prefill(i):
    c = PREFILL[i]
    x = draw(c, i)
    err = torch.zeros(1, dtype=i32, device="cuda")
    o, pool = run(c, x, err_flag=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    compare(c, x, o, pool)


def test_prefill_of_many_sequences():
    """More sequences than a warp has lanes, of 0 to 9 tokens, and with two long ones
    among them; each against itself alone."""
    gen = torch.Generator().manual_seed(40)
    lengths = torch.randint(0, 10, (150,), generator=gen).tolist()
    for more in ((), (700, 1500)):
        lengths[60:60 + len(more)] = more
        c = case(lengths, H=2, gate="fixed")
        x = draw(c, 41)
        err = torch.zeros(1, dtype=i32, device="cuda")
        o, pool = run(c, x, err_flag=err)
        assert err.item() == 0
        some = [0, 1, 31, 32, 60, 61, 62, 63, 64, 100, 149]
        for n in some:
            s = slice(int(x["cu"][n]), int(x["cu"][n + 1]))
            if s.start == s.stop:
                continue
            y = dict(x, cu=torch.tensor([0, lengths[n]], dtype=i32), idx=x["idx"][n:n + 1], **{k: x[k][s] for k in "qkv"})
            compare(dict(c, lengths=[lengths[n]]), y, o[s], pool, others=False)
        rest = [k for k in range(len(pool)) if k not in x["idx"].tolist()]
        assert torch.equal(pool[rest].cpu(), x["pool"][rest])


def test_prefill_fixed_layout_equals_cu_seqlens():
    c = case([70, 70, 70], H=2)
    x = draw(c, 50)
    want = run(c, x)
    up = {k: v.cuda() for k, v in x.items()}
    o = torch.empty_like(want[0])
    kda.kda_lin_prefill(lu.dims(c), lu.scalar_gate(x["A_log"], x["dt_bias"], True), up["q"], up["k"], up["v"], up["a"], up["pool"],
                        up["idx"], None, 3, o)
    assert torch.equal(o, want[0]) and torch.equal(up["pool"], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prefill_padding_and_bad_slots(dtype):
    """A sequence of slot -1 or of no slot gets zero outputs; the others what they
    get alone."""
    c = case([100, 40, 70, 30], H=1, HV=2, dtype=dtype)
    x = draw(c, 60)
    good = run(c, x)
    for bad, bit in ((-1, 0), (7, kda.KDA_DEVERR_SLOT), (-2, kda.KDA_DEVERR_SLOT)):
        y = dict(x, idx=x["idx"].clone())
        y["idx"][1] = bad
        err = torch.zeros(1, dtype=i32, device="cuda")
        o, pool = run(c, y, err_flag=err)
        assert err.item() == bit
        assert not o[100:140].any()
        keep = torch.ones(len(o), dtype=torch.bool)
        keep[100:140] = False
        assert torch.equal(o[keep], good[0][keep])
        slot = int(x["idx"][1])
        assert torch.equal(pool[slot].cpu(), x["pool"][slot])
        rest = [s for s in range(7) if s != slot]
        assert torch.equal(pool[rest], good[1][rest])


@pytest.mark.parametrize("cu", [[0, 50, 40, 120], [0, 50, 130, 120], [1, 50, 60, 120], [0, 50, 60, 119], [0, -4, 60, 120]])
def test_prefill_bad_bounds(cu):
    """Bounds that are none are flagged; sequences with bounds of their own still run
    and nothing else is written."""
    c = case([50, 10, 60], H=1)
    x = dict(draw(c, 61), cu=torch.tensor(cu, dtype=i32))
    err = torch.zeros(1, dtype=i32, device="cuda")
    o, pool = run(c, x, err_flag=err)
    assert err.item() == kda.KDA_DEVERR_SEQLENS
    free = [s for s in range(6) if s not in x["idx"].tolist()]
    assert torch.equal(pool[free].cpu(), x["pool"][free])


@pytest.mark.parametrize("n,T", [(7, 2000), (40, 4000), (9, 64)])
def test_prefill_of_overlapping_sequences(n, T):
    """Bounds that go back and forth: flagged, nothing runs, and nothing is written past
    the workspace."""
    c = case([T], H=1, gate="given")
    x = draw(c, 63, spare=n)
    x.update(cu=torch.tensor([T * (i & 1) for i in range(n)] + [T], dtype=i32), idx=torch.arange(n, dtype=i32))
    size = kda.kda_lin_prefill_workspace_size(lu.dims(c), n, T)
    ws = torch.full((size + 2 ** 20,), 77, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=i32, device="cuda")
    o, pool = run(dict(c, lengths=[0] * n), x, err_flag=err, workspace=ws[:max(size, 1)])
    assert err.item() == kda.KDA_DEVERR_SEQLENS and (o == 7).all() and torch.equal(pool.cpu(), x["pool"]) and (ws == 77).all()


SIZES = [(1, 128, 4), (1, 4096, 16), (8, 16980, 2), (64, 16384, 4), (200, 9000, 8), (16, 16, 64), (3, 764, 2), (2, 9000, 1),
         (5, 4001, 7), (33, 10000, 3)]


@pytest.mark.parametrize("n,T,HV", SIZES)
def test_prefill_workspace_holds_every_cut(n, T, HV):
    """Lengths of every kind keep within the workspace, and the longest sequence ends where
    it ends without a cut."""
    import random

    size = kda.kda_lin_prefill_workspace_size(kda.dims(HV), n, T)
    rng = random.Random(n * T)
    d = lu.dims(case([T], H=1, HV=HV))
    for kind in range(6):
        w = [rng.random() ** (kind * 2) + (1e-3 if kind < 4 else 0) for _ in range(n)]
        if kind == 5:
            w = [1.0] + [0.0] * (n - 1)
        lengths = [int(T * x / sum(w)) for x in w]
        lengths[rng.randrange(n)] += T - sum(lengths)
        ws = torch.full((size + 2 ** 18,), 77, dtype=torch.uint8, device="cuda")
        c = case(lengths, H=1, HV=HV, gate="fixed")
        x = draw(c, kind)
        err = torch.zeros(1, dtype=i32, device="cuda")
        o, pool = run(c, x, err_flag=err, workspace=ws[:max(size, 1)])
        assert err.item() == 0 and (ws[size:] == 77).all()
        at = max(range(n), key=lambda i: lengths[i])  # the longest, alone and uncut, in parts of 64
        s0 = sum(lengths[:at])
        idx, L, end = x["idx"][at:at + 1].cuda(), lengths[at], s0 + lengths[at]
        parts = {}
        for name, f in (("state", lambda t: t.cuda()), ("magnitude", lambda t: t.abs().cuda())):
            q, k, v, parts[name] = (f(x[key]) for key in ("q", "k", "v", "pool"))
            for t in range(s0, end, 64):
                e = min(t + 64, end)
                kda.kda_lin_prefill(d, lu.scalar_gate(x["A_log"], None, True), q[t:e], k[t:e], v[t:e], None, parts[name], idx, None, 1,
                                    torch.empty_like(v[t:e]))
        # the same terms, in another order: 2^-24 of the magnitudes' sum for each of the at most
        # 64 additions and 3 products of a chunk's, and for a product and a sum a chunk, twice
        bound = (2 * 67 + 4 * (L // 64 + 1)) * 2.0 ** -24 * parts["magnitude"][idx.long()]
        assert ((pool[idx.long()] - parts["state"][idx.long()]).abs() <= bound).all()
        assert torch.isfinite(o[s0:end]).all() and not (o[s0:end] == 7).all(-1).any()


def test_prefill_nan_stays_in_its_sequence():
    c = case([90, 66, 130], H=2)
    x = draw(c, 62)
    good = run(c, x)
    for name in "qkv":
        y = dict(x, **{name: x[name].clone()})
        y[name][90:156] = float("nan")
        o, pool = run(c, y)
        for s, n in ((slice(0, 90), 0), (slice(156, 286), 2)):
            slot = int(x["idx"][n])
            assert torch.equal(o[s], good[0][s]) and torch.equal(pool[slot], good[1][slot])
    # the chunks before a bad token are as they were
    y = dict(x, v=x["v"].clone())
    y["v"][156 + 100] = float("inf")
    o, _ = run(c, y)
    assert torch.equal(o[156:156 + 64], good[0][156:156 + 64])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prefill_in_parts(dtype):
    """Two calls, the second from the state of the first, against the rule over both."""
    c = case([300], H=1, HV=2, dtype=dtype, gate="fixed")
    x = draw(c, 63, pad=0)
    pool = x["pool"].cuda()
    o = torch.empty(300, 2, V, dtype=lu.DT[dtype], device="cuda")
    for s in (slice(0, 101), slice(101, 300)):
        q, k, v = (x[n][s].cuda() for n in "qkv")
        kda.kda_lin_prefill(lu.dims(c), lu.scalar_gate(x["A_log"], None, True), q, k, v, None, pool, x["idx"].cuda(), None, 1, o[s])
    compare(c, x, o, pool, parts=(0, 101))


def test_prefill_captured_and_on_another_stream():
    c = case([200, 500, 64], H=2, HV=4)
    x = draw(c, 64)
    want = run(c, x)
    up = {k: v.cuda() for k, v in x.items()}
    start = up["pool"].clone()
    o = torch.zeros_like(want[0])
    gate = lu.scalar_gate(x["A_log"], x["dt_bias"], True)
    ws = torch.empty(max(1, kda.kda_lin_prefill_workspace_size(lu.dims(c), 3, 764)), dtype=torch.uint8, device="cuda")
    call = lambda **kw: kda.kda_lin_prefill(lu.dims(c), gate, up["q"], up["k"], up["v"], up["a"], up["pool"], up["idx"],  # noqa: E731
                                            up["cu"], 3, o, **kw)
    graphs = []
    for _ in range(2):  # two graphs share a workspace
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(workspace=ws)
    for g in graphs + graphs[:1]:
        up["pool"].copy_(start)
        o.zero_()
        ws.fill_(0xff)
        g.replay()
        assert torch.equal(o, want[0]) and torch.equal(up["pool"], want[1])
    up["pool"].copy_(start)
    o.zero_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(o, want[0]) and torch.equal(up["pool"], want[1])


def test_prefill_of_aligned_views():
    """q, k, v, o and the pool inside larger tensors, 16 bytes off."""
    c = case([150, 33], H=1, HV=2)
    x = draw(c, 65)
    want = run(c, x)
    up = {k: v.cuda() for k, v in x.items()}
    for n in "qkv":
        big = torch.full((up[n].numel() + 8,), float("nan"), dtype=up[n].dtype, device="cuda")
        big[8:] = up[n].flatten()
        up[n] = big[8:].view(up[n].shape)
    states = torch.full((up["pool"].numel() + 4,), 3.0, device="cuda")  # a pool that is aligned to 16 bytes and no more
    states[4:] = up["pool"].flatten()
    up["pool"] = states[4:].view(up["pool"].shape)
    big = torch.full((want[0].numel() + 16,), 3.0, dtype=want[0].dtype, device="cuda")
    o = big[8:-8].view(want[0].shape)
    kda.kda_lin_prefill(lu.dims(c), lu.scalar_gate(x["A_log"], x["dt_bias"], True), up["q"], up["k"], up["v"], up["a"], up["pool"],
                        up["idx"], up["cu"], 2, o)
    assert torch.equal(o, want[0]) and torch.equal(up["pool"], want[1])
    assert (big[:8] == 3).all() and (big[-8:] == 3).all() and (states[:4] == 3).all()


def packed(c, x):
    return torch.cat([x[n].flatten(1) for n in "qkv"], 1)


STEP = [case([1] * 3, H=2, HV=4), case([1], dtype="f16", gate="fixed", norm=False), case([1] * 40, H=4, HV=16, gate="given"),
        case([1] * 5, H=1, HV=3, dtype="f16", gate="strong"), case([1] * 2, gate="out")]


@pytest.mark.parametrize("i", range(len(STEP)))
def test_decode(i):
    c = STEP[i]
    B = len(c["lengths"])
    x = draw(c, 100 + i, pad=0)
    rows = packed(c, x)
    wide = torch.full((B, rows.shape[1] + 16), 9.0, dtype=rows.dtype)  # a row stride of its own
    wide[:, :rows.shape[1]] = rows
    pool, idx = x["pool"].cuda(), x["idx"].clone()
    if B > 1:
        idx[1] = -1
    o = torch.full((B, c["HV"], V), 7.0, dtype=rows.dtype, device="cuda")
    err = torch.zeros(1, dtype=i32, device="cuda")
    kda.kda_lin_decode_packed(lu.dims(c), lu.scalar_gate(x["A_log"], x["dt_bias"], c["norm"]), wide.cuda()[:, :rows.shape[1]],
                              None if x["a"] is None else x["a"].cuda(), pool, idx.cuda(), o, err_flag=err)
    assert err.item() == 0
    if B > 1:
        assert not o[1].any()
        slot = int(x["idx"][1])
        assert torch.equal(pool[slot].cpu(), x["pool"][slot])
    g = so.lin_decay(B, lu.host(x["a"]), lu.host(x["A_log"]), lu.host(x["dt_bias"]))
    for r in range(B):
        if idx[r] < 0:
            continue
        S0 = lu.host(x["pool"][idx[r]])
        q, k, v = (lu.host(x[n][r:r + 1]) for n in "qkv")
        o_ref, states = so.lin_sequence(S0, q, k, v, g[r:r + 1], SCALE, c["norm"])
        o_b, s_b = lu.bounds(S0, q, k, v, g[r:r + 1], SCALE, c["norm"], c["dtype"], exact_weights=True)
        lu.check("o", o[r], o_ref[0], o_b[0], c["dtype"])
        lu.check("state", pool[idx[r]], states[0], s_b)


VERIFY = [(2, 6, False, case([], H=2, HV=4)), (1, 1, False, case([], dtype="f16")), (3, 5, True, case([], H=1, HV=2, gate="fixed", norm=False)),
          (2, 40, True, case([], dtype="f16", gate="given")), (12, 3, False, case([], H=4, HV=8, gate="strong"))]


@pytest.mark.parametrize("i", range(len(VERIFY)))
def test_verify_and_commit(i):
    B, T, tree, c = VERIFY[i]
    c = dict(c, lengths=[T] * B)
    x = draw(c, 200 + i, pad=0)
    gen = torch.Generator().manual_seed(i)
    parent = None
    if tree:
        parent = torch.stack([torch.cat([torch.randint(-1, max(t, 1), (1,), generator=gen) if t else torch.tensor([-1])
                                         for t in range(T)]) for _ in range(B)]).int()
    idx = x["idx"].clone()
    if B > 1:
        idx[1] = -1
    pool = x["pool"].cuda()
    o = torch.full((B, T, c["HV"], V), 7.0, dtype=lu.DT[c["dtype"]], device="cuda")
    snaps = torch.full((B, T, c["HV"], V, K), 5.0, device="cuda")
    gate, a = lu.scalar_gate(x["A_log"], x["dt_bias"], c["norm"]), None if x["a"] is None else x["a"].cuda()
    args = (lu.dims(c), gate, packed(c, x).cuda(), a, B, T)
    if tree:
        kda.kda_lin_verify_tree(*args, parent.cuda(), pool, idx.cuda(), o, snaps)
    else:
        kda.kda_lin_verify_chain(*args, pool, idx.cuda(), o, snaps)
    assert torch.equal(pool.cpu(), x["pool"])
    g = so.lin_decay(B * T, lu.host(x["a"]), lu.host(x["A_log"]), lu.host(x["dt_bias"]))
    for r in range(B):
        if idx[r] < 0:
            assert not o[r].any() and (snaps[r] == 5).all()
            continue
        s = slice(r * T, r * T + T)
        S0 = lu.host(x["pool"][idx[r]])
        q, k, v = (lu.host(x[n][s]) for n in "qkv")
        par = parent[r].tolist() if tree else list(range(-1, T - 1))
        o_ref, states = so.lin_sequence(S0, q, k, v, g[s], SCALE, c["norm"], par)
        for t in range(T):  # the bound of a node is that of its path
            path = [t]
            while par[path[0]] >= 0:
                path.insert(0, par[path[0]])
            o_b, s_b = lu.bounds(S0, q[path], k[path], v[path], g[s][path], SCALE, c["norm"], c["dtype"], exact_weights=True)
            lu.check("o", o[r, t], o_ref[t], o_b[-1], c["dtype"])
            lu.check("snapshot", snaps[r, t], states[t], s_b)
    accepted = torch.tensor([T - 1] + [-1] * (B - 1), dtype=i32)
    kda.kda_commit(lu.dims(c), snaps, B, T, accepted.cuda(), pool, idx.cuda())
    assert torch.equal(pool[idx[0]], snaps[0, T - 1])


def test_verify_refuses_bad_parents_and_slots():
    c = case([3] * 3)
    x = draw(c, 300, pad=0)
    parent = torch.tensor([[-1, 0, 2], [-1, -2, 0], [-1, 0, 1]], dtype=i32)
    o = torch.full((3, 3, 1, V), 7.0, dtype=torch.bfloat16, device="cuda")
    snaps = torch.full((3, 3, 1, V, K), 5.0, device="cuda")
    err = torch.zeros(1, dtype=i32, device="cuda")
    args = (lu.dims(c), lu.scalar_gate(x["A_log"], x["dt_bias"], True), packed(c, x).cuda(), x["a"].cuda(), 3, 3)
    kda.kda_lin_verify_tree(*args, parent.cuda(), x["pool"].cuda(), x["idx"].cuda(), o, snaps, err_flag=err)
    assert err.item() == kda.KDA_DEVERR_PARENT
    assert not o[:2].any() and (snaps[:2] == 5).all() and o[2].any()
    err.zero_()
    kda.kda_lin_verify_chain(*args, x["pool"].cuda(), torch.tensor([6, -5, 0], dtype=i32, device="cuda"), o, snaps, err_flag=err)
    assert err.item() == kda.KDA_DEVERR_SLOT and not o[:2].any()


def test_prefill_then_decode_is_one_longer_prefill():
    """The state that a prefill leaves is the one that decode goes on from."""
    c = case([129], H=1, HV=2)
    x = draw(c, 310, pad=0)
    o, pool = run(c, x)
    first = dict(x, cu=torch.tensor([0, 128], dtype=i32), **{n: x[n][:128] for n in "qkv"}, a=x["a"][:128])
    _, pool2 = run(dict(c, lengths=[128]), first)
    last = torch.cat([x[n][128:].flatten(1) for n in "qkv"], 1).cuda()
    o2 = torch.empty(1, 2, V, dtype=torch.bfloat16, device="cuda")
    kda.kda_lin_decode_packed(lu.dims(c), lu.scalar_gate(x["A_log"], x["dt_bias"], True), last, x["a"][128:].cuda(), pool2,
                              x["idx"].cuda(), o2)
    compare(c, x, torch.cat([o[:128], o2]), pool2)
