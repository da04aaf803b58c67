"""Inputs, the FP64 oracle's answers and error bounds for linear attention with
one decay per value head.

Bounds, element by element, from sums of magnitudes.  With u the half step of
the 16-bit type (BF16 2^-8, FP16 2^-11 relative to the value):
  - an output is rounded once: u |o|, and FP16 numbers below 2^-14 lie 2^-24 apart,
    so that their rounding is off by up to 2^-25 whatever u |o| is;
  - inside a chunk the weights q.k e^(..) of the values are rounded once to 16
    bits: u (1 + u) scale sum_j |q.k_j| e^(c_i - c_j) |v_j|.  FP16 weights are kept times a power of two that takes
    |q_i| max_j |k_j| above 2^14, with steps of 2^-24 at the bottom, 2^-38 of that:
    2^-39 scale |q_i| max_j |k_j| sum_j |v_j|;
  - for its product with q the state before a chunk is rounded once to 16 bits:
    u (1 + u) scale e^(c_i) sum_k |q_k| |S_vk|;
  - everything else is FP32 or a pair of 16-bit halves: exponentials 2^-17 for the
    smallest factors, norms 2^-22, halves 2^-17, sums of 64 and 128 terms 2^-16.4
    of the magnitudes' sum, all told below 2^-14 of scale |q|.(|S| built from
    magnitudes).  As a factor of FP16's a row of the state is kept likewise: 2^-39 of
    its largest, 2^-39 |q|_1 max_k |S_vk|.
  - states: 2^-14 of the sum of magnitudes.  FP16 parts of a decayed key end 2^-24
    apart: off by up to 2^-25 whatever the decay inside the chunk of 64 tokens has left
    of it (unit keys are taken times 2^15: 2^-40).  That adds 2^-25 sum |v_j| a chunk,
    which then decays with the state, and |q|_1 of it to an output."""
import numpy as np
import torch

from linear_attention_serving_gated_gb300 import kda
from oracle import serving_oracle as so

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
REST = 2.0 ** -14


def dims(c):
    return kda.dims(c["H"], HV=c["HV"], dtype=kda.KDA_DTYPE_F16 if c["dtype"] == "f16" else kda.KDA_DTYPE_BF16)


def gate_inputs(gen, gate, rows, HV, dt):
    """(A_log, dt_bias, a), on the CPU."""
    if gate == "fixed":
        return -torch.rand(HV, generator=gen) * 5, None, None
    if gate == "none":  # a state that keeps everything
        return None, None, torch.zeros(rows, HV)
    if gate in ("given", "strong", "out"):
        a = -torch.rand(rows, HV, generator=gen) ** 3 * 2
        if gate != "given":  # some tokens forget everything, and some log-decays are no such thing
            kind = torch.randint(0, 12, (rows, HV), generator=gen)
            a = torch.where(kind == 0, -60.0, torch.where(kind == 1, -1e9, torch.where(kind == 2, -128.0, a)))
            if gate == "out":
                a = torch.where(kind == 3, 5.0, torch.where(kind == 4, -torch.inf, a))
        return None, None, a
    A_log = torch.log(torch.rand(HV, generator=gen) * 15 + 1)
    return A_log, torch.randn(HV, generator=gen) - 4 if gate == "raw" else None, torch.randn(rows, HV, generator=gen).to(dt)


def scalar_gate(A_log, dt_bias, norm, scale=128 ** -0.5):
    up = lambda x: None if x is None else x.cuda()  # noqa: E731
    return kda.ScalarGate(A_log=up(A_log), dt_bias=up(dt_bias), use_qk_l2norm=norm, scale=scale)


def host(x):
    return None if x is None else x.double().numpy()


def bounds(S0, q, k, v, g, scale, norm, dtype, exact_weights=False, parts=(0,)):
    """Error bounds of (outputs [T,HV,V], last state) of one sequence, prefilled in
    parts that start at the given tokens."""
    G = v.shape[1] // q.shape[1]
    q, k = (np.repeat(so.lin_unit(x, norm), G, 1) for x in (q, k))
    X, signed = np.asarray(S0, np.float64), np.asarray(v, np.float64)  # the state itself
    v = np.abs(signed)
    T = len(q)
    c = np.cumsum(g, 0)
    S = np.abs(np.asarray(S0, np.float64))
    step = 0.0 if dtype != "f16" or exact_weights else 2.0 ** -40 if norm else 2.0 ** -25
    E, E0 = np.zeros(v.shape[1:]), np.zeros(v.shape[1:])  # of a state's rows; at the chunk's start
    o = np.zeros(v.shape)
    for t in range(T):
        S = np.exp(g[t])[:, None, None] * S + v[t][:, :, None] * np.abs(k[t])[:, None, :]
        aq = np.abs(q[t])
        if (t - max(x for x in parts if x <= t)) % 64 == 0:  # a chunk starts
            E0, c0 = E, c[t - 1] if t else 0 * c[0]
            X0, mine = np.abs(X), 0 * E
        X = np.exp(g[t])[:, None, None] * X + signed[t][:, :, None] * k[t][:, None, :]
        mine = mine + step * v[t]
        E = np.exp(c[t] - c0)[:, None] * E0 + mine
        o[t] = scale * (REST * np.einsum("hvk,hk->hv", S, aq) + E0 * aq.sum(-1)[:, None])
        if not exact_weights:
            u = U[dtype]
            o[t] += u * (1 + u) * scale * np.exp(c[t] - c0)[:, None] * np.einsum("hvk,hk->hv", X0, aq)
        if dtype == "f16":
            o[t] += 2.0 ** -39 * scale * aq.sum(-1)[:, None] * S.max(-1)
    if not exact_weights:
        u = U[dtype]
        for h in range(v.shape[1]):
            with np.errstate(over="ignore"):
                w = scale * np.abs(q[:, h] @ k[:, h].T) * np.tril(np.exp(np.minimum(c[:, None, h] - c[None, :, h], 0)))
            o[:, h] += u * (1 + u) * (w @ v[:, h])
            if dtype == "f16":
                norm_of = lambda x: np.sqrt((x * x).sum(-1))  # noqa: E731
                o[:, h] += 2.0 ** -39 * scale * (norm_of(q[:, h]) * norm_of(k[:, h]).max())[:, None] * np.cumsum(v[:, h], 0)
    return o, REST * S + E[:, :, None]


def check(what, got, ref, bound, dtype=None):
    got = got.detach().double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: not finite"
    bound = bound + (U[dtype] * np.abs(ref) if dtype else 0) + (2.0 ** -25 if dtype == "f16" else 1e-30)
    worst = np.max(np.abs(got - ref) / bound) if ref.size else 0.0
    assert worst <= 1, f"{what}: {worst:.3f} of its bound"
