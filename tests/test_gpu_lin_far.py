"""Linear attention and the archive where offsets pass 2^31 and 2^32 elements."""
import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so
from tests import lin_util as lu

pytestmark = pytest.mark.gpu
K = V = 128
HV, SCALE = 64, K ** -0.5
HEADS = [0, 63]
i32 = torch.int32


def gpu(*shape, dt=torch.bfloat16):
    return torch.randn(*shape, device="cuda", dtype=dt)


def near(what, got_o, got_s, S0, q, k, v, A_log, exact=False):
    """Outputs [T,2,V] and states [T or 1,2,V,K] of the two heads against the oracle."""
    g = so.lin_decay(len(q), None, lu.host(A_log.cpu()[HEADS]), None)
    S0, q, k, v = (lu.host(x.cpu()) for x in (S0, q, k, v))
    o_ref, states = so.lin_sequence(S0, q, k, v, g, SCALE)
    o_b, s_b = lu.bounds(S0, q, k, v, g, SCALE, True, "bf16", exact_weights=exact)
    lu.check(f"o of {what}", got_o, o_ref, o_b, "bf16")
    lu.check(f"state of {what}", got_s, states[-1], s_b)


def test_far_tokens_slots_and_snapshots():
    torch.manual_seed(1)
    d, slots, tail = kda.dims(1, HV=HV), 4200, 164
    A_log = -torch.rand(HV, device="cuda") * 5
    gate = kda.ScalarGate(A_log=A_log)
    pool = torch.zeros(slots, HV, V, K, device="cuda")  # 2^32 elements and more
    pool[-2:] = gpu(2, HV, V, K, dt=torch.float32) * 0.3
    start = pool[-2:].clone()
    T = 2 ** 19 + 200  # outputs past 2^32 elements
    q, k, v = gpu(T, 1, K), gpu(T, 1, K), gpu(T, HV, V)
    o, err = torch.empty_like(v), torch.zeros(1, dtype=i32, device="cuda")
    kda.kda_lin_prefill(d, gate, q, k, v, None, pool, torch.tensor([0, slots - 1], dtype=i32, device="cuda"),
                        torch.tensor([0, T - tail, T], dtype=i32, device="cuda"), 2, o, err_flag=err)
    near("the last tokens", o[-tail:, HEADS], pool[-1, HEADS], start[1, HEADS], q[-tail:], k[-tail:], v[-tail:, HEADS], A_log)
    del o, v

    row = gpu(1, 2 * K + HV * V)
    parts = row[:, :K].view(1, 1, K), row[:, K:2 * K].view(1, 1, K), row[:, 2 * K:].view(1, HV, V)[:, HEADS]
    out, idx = torch.empty(1, HV, V, dtype=torch.bfloat16, device="cuda"), torch.tensor([slots - 2], dtype=i32, device="cuda")
    kda.kda_lin_decode_packed(d, gate, row, None, pool, idx, out, err_flag=err)
    near("a far slot", out[:, HEADS], pool[-2, HEADS], start[0, HEADS], *parts, A_log, exact=True)

    pool[-2] = start[0]
    B, steps = 2100, 2
    rows = torch.zeros(B * steps, row.shape[1], dtype=torch.bfloat16, device="cuda")
    rows[-2:] = gpu(2, row.shape[1])
    q, k, v = rows[-2:, :K].view(2, 1, K), rows[-2:, K:2 * K].view(2, 1, K), rows[-2:, 2 * K:].view(2, HV, V)[:, HEADS]
    idx = torch.full((B,), slots - 2, dtype=i32, device="cuda")
    out = torch.empty(B * steps, HV, V, dtype=torch.bfloat16, device="cuda")
    snaps = torch.empty(B, steps, HV, V, K, device="cuda")
    kda.kda_lin_verify_chain(d, gate, rows, None, B, steps, pool, idx, out, snaps, err_flag=err)
    near("a far snapshot", out[-2:, HEADS], snaps[-1, -1, HEADS], start[0, HEADS], q, k, v, A_log, exact=True)
    assert err.item() == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_far_pages(bits):
    torch.manual_seed(2)
    slots = 1 << (12 if bits == 8 else 13)  # codes past 2^32 bytes
    pool = torch.zeros(1, 4200, HV, V, K, device="cuda")
    pool[0, -1] = gpu(HV, V, K, dt=torch.float32)
    codes = torch.empty(slots + 8, 1, HV, V, K if bits == 8 else K // 2, dtype=torch.int8 if bits == 8 else torch.uint8, device="cuda")
    scales = torch.empty(slots + 8, 1, HV, V, 1 if bits == 8 else 4, device="cuda")
    near, far, last = (torch.tensor([x], dtype=i32, device="cuda") for x in (0, slots + 7, 4199))
    for page in (near, far):
        kda.kda_pool_store(pool, codes, scales, last, page)
    assert torch.equal(codes[0], codes[-1]) and torch.equal(scales[0], scales[-1]) and codes[-1].any()
    want = pool[0, -1].clone()
    pool[0, -1] = 0
    kda.kda_pool_load(codes, scales, pool, far, last)
    off = (pool[0, -1] - want).abs().max().item()
    assert 0 < off <= want.abs().max().item() / (254 if bits == 8 else 14) * (1 + 2.0 ** -20)
    assert np.isfinite(off)
