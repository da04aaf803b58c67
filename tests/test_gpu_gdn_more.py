"""The per-head gated delta rule where its other tests do not go: deep trees, keys
that share a direction, and FP16 outputs held to FP16's own rounding."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from tests.gpu_util import assert_o_close, assert_s_close, host_f64, rms
from tests.test_gpu_gdn import K, assert_state, f64, gate_of, make, oracle_rows, packed_of, prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H,HV,f16", [(2, 33, 1, 2, False), (1, 70, 2, 2, False), (2, 70, 1, 2, True), (40, 34, 1, 8, False)])
def test_trees_of_more_than_32_nodes(B, T, H, HV, f16):
    """Parents on both sides of node 32, several children of one node above it."""
    d = make(20, B * T, H, HV, B + 1, f16=f16)
    rng = np.random.default_rng(T)
    parents = np.array([[int(rng.integers(-1, i)) for i in range(T)] for _ in range(B)], np.int32)
    parents[0, 33:] = 32  # all children of one node
    if T > 40:
        parents[-1, 35:40], parents[-1, 40:] = [31, 32, 33, 31, 32], np.maximum(parents[-1, 40:], 30)
    pool = d["pool"].cuda()
    o = torch.zeros(B, T, HV, K, dtype=d["dt"], device="cuda")
    snap = torch.zeros(B, T, HV, K, K, device="cuda")
    args = (d["dims"], gate_of(d), packed_of(d, B * T).cuda(), d["a"].cuda(), d["b"].cuda(), B, T)
    idx = d["idx"][:B].cuda()
    kda.kda_gdn_verify_tree(*args, torch.from_numpy(parents).cuda(), pool, idx, o, snap)
    assert torch.equal(pool.cpu(), d["pool"])
    for r in sorted({0, B // 2, B - 1}):
        out, st = oracle_rows(d, slice(r * T, (r + 1) * T), f64(d["pool"][d["idx"][r]]), parents[r])
        assert_o_close(o[r], out)
        assert_state(snap[r], st, 2.0 ** -18 * (T + 1) * np.abs(st).max())
    # a parent that is none, past node 32, refuses its request alone
    bad = parents.copy()
    bad[0, T - 1] = T - 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o2, snap2 = torch.full_like(o, 3.0), torch.full_like(snap, 3.0)
    kda.kda_gdn_verify_tree(*args, torch.from_numpy(bad).cuda(), pool, idx, o2, snap2, err_flag=err)
    assert int(err) == kda.KDA_DEVERR_PARENT
    assert bool((o2[0] == 0).all()) and bool((snap2[0] == 3).all())
    assert torch.equal(o2[1:], o[1:]) and torch.equal(snap2[1:], snap[1:])


def oracle_prefill(d, lengths):
    outs, pool, t0 = [], f64(d["pool"]).copy(), 0
    for n, L in enumerate(lengths):
        if L:
            out, states = oracle_rows(d, slice(t0, t0 + L), pool[int(d["idx"][n])])
            outs.append(out)
            pool[int(d["idx"][n])] = states[-1]
        t0 += L
    return np.concatenate(outs), pool


LENGTHS = [[700], [300, 70], [40, 130, 1, 64, 65, 200] * 4, [30] * 80]  # thinnest to wide


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("slow", [False, True])
def test_fp16_outputs_within_their_own_rounding(lengths, slow):
    """An FP16 output is off by half a step, 2^-11 of its value.  What the state
    and the products lose stays below a half of that: five operands (S, T, Y, D,
    P) keep 2^-18 each, and Q S and P D, which may cancel, are up to 10 times the
    output."""
    d = make(21, sum(lengths), 2, 4, len(lengths) + 1, f16=True, given=slow)
    if slow:
        d["a"] = -torch.rand(sum(lengths), 4) * 1e-3
    o, pool = prefill(d, lengths)
    want, _ = oracle_prefill(d, lengths)
    assert rms(host_f64(o) - want) <= (2.0 ** -11 + 2.0 ** -12) * rms(want)


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("slow", [False, True])
def test_keys_that_share_a_direction(lengths, f16, slow):
    """Keys and queries 0.9 along one direction and beta near 1, as in layers of
    trained models: what a token writes, the next ones take back.  The inverse's
    entries and with them the rounding of its operands are larger than for
    independent keys; states are held to the framework's bound for FP32 states."""
    T = sum(lengths)
    d = make(22, T, 2, 4, len(lengths) + 1, f16=f16, given=slow)
    if slow:
        d["a"] = -torch.rand(T, 4) * 1e-3
    g = torch.Generator().manual_seed(5)
    common = torch.randn(2, K, generator=g)
    for n in ("q", "k"):
        d[n] = (0.9 ** 0.5 * common + 0.1 ** 0.5 * torch.randn(T, 2, K, generator=g)).to(d["dt"])
    d["b"] = (torch.randn(T, 4, generator=g) + 3).to(d["dt"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, pool = prefill(d, lengths, err=err)
    want, ref_pool = oracle_prefill(d, lengths)
    assert int(err) == 0
    assert_o_close(o, want)
    got = host_f64(pool)
    for n in range(len(lengths)):
        s = int(d["idx"][n])
        assert_s_close(got[s], ref_pool[s])


@pytest.mark.parametrize("seqs", [1, 80])  # thinnest, wide
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_decay_alone_is_that_of_decode(seqs, f16, given):
    """Sequences of one token with beta 0: the state times the decay's factor, the
    same FP32 product as a decode's, bit for bit."""
    d = make(23, seqs, 1, 4, seqs, f16=f16, given=given, raw_beta=False)
    d["b"][:] = 0
    if given:
        d["a"] = -torch.linspace(0.0, 80.0, seqs * 4).view(seqs, 4).flip(1).contiguous()
    _, pool = prefill(d, [1] * seqs)
    other, o = d["pool"].cuda(), torch.zeros(seqs, 4, K, dtype=d["dt"], device="cuda")
    kda.kda_gdn_decode_packed(d["dims"], gate_of(d), packed_of(d, seqs).cuda(), d["a"].cuda(), d["b"].cuda(), other,
                              d["idx"].cuda(), o)
    assert torch.equal(pool, other)
