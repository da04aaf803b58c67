"""Cases and plain forms of the calls that join the serving operators: linear
attention with one decay per head (chunked prefill, packed decode, chain and
tree verify), the log probabilities of given tokens with entropy and top
alternatives, and pages of a state pool stored in 8 or 4 bits and read back.

`own` selects what `run` computes with: False, elementary torch operations;
True, the library's entry points.

The rule, per value head, S a K x V state, one log-decay g_t per token:
    S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
    g_t = -exp(A_log) softplus(a_t + dt_bias), or given, or the head's own
          -exp(A_log) for every token
    q, k divided by sqrt(sum x^2 + 1e-6), or as they are
"""
import math

import torch

own = False

K = V = 128
CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GROUP = {8: 128, 4: 32}  # values that share a scale
TOP = {8: 127, 4: 7}  # the largest code


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one short prompt of a small model: latency counts
        dict(name="prefill_1x128_h4", op="prefill", lengths="128", H=4, HV=4, slots=4, pad=0, dtype="bf16", gate="raw", norm=True),
        # one prompt of the framework's headline length and heads
        dict(name="prefill_1x4096_h16", op="prefill", lengths="4096", H=16, HV=16, slots=16, pad=0, dtype="bf16", gate="raw", norm=True),
        # a scheduler's step over a ragged batch padded to a 32768-row bucket, heads of fixed decay
        dict(name="prefill_varlen8_h16", op="prefill", lengths="1,8087,517,2048,1290,3331,64,1642", H=16, HV=16, slots=240,
             pad=32768 - 16980, dtype="bf16", gate="fixed", norm=False),
        # grouped value heads, FP16 tokens, log-decays given in FP32, odd lengths
        dict(name="prefill_ragged_f16_h8_hv16", op="prefill", lengths="1000,333,77,2001", H=8, HV=16, slots=16, pad=5,
             dtype="f16", gate="given", norm=True),
        # one user generating: the smallest decode step
        dict(name="decode_1_h16", op="decode", B=1, H=16, HV=16, slots=240, dtype="bf16", gate="raw", norm=True),
        # a full decode batch with grouped value heads
        dict(name="decode_48_h16_hv32", op="decode", B=48, H=16, HV=32, slots=240, dtype="bf16", gate="raw", norm=True),
        # speculative verify of six tokens for sixteen requests, state snapshots kept
        dict(name="verify_16x6_h16", op="verify", B=16, T=6, tree=False, H=16, HV=16, slots=240, dtype="bf16", gate="raw", norm=True),
        # draft trees of a few requests, FP16, heads of fixed decay
        dict(name="verify_tree_4x10_f16_h8", op="verify", B=4, T=10, tree=True, H=8, HV=8, slots=240, dtype="f16", gate="fixed", norm=False),
        # one request's drafts under a grammar that masks most of an odd vocabulary, few alternatives asked
        dict(name="logprobs_6x50257_f16", op="logprobs", rows=6, vocab=50257, top=5, pad=0, masked=True, idle=False, dtype="f16"),
        # every row of a full batch of drafts against a large vocabulary, the usual most of alternatives
        dict(name="logprobs_288x131072", op="logprobs", rows=288, vocab=131072, top=20, pad=0, masked=False, idle=True, dtype="f32"),
        # a small model's two finished requests kept for later in 4 bits, and taken up again
        dict(name="archive_2_of_16_h4_4bit", op="archive", layers=1, slots=16, heads=4, rows=2, bits=4),
        # a full pool: a third of the pages of four layers kept in 8 bits and read back
        dict(name="archive_70_of_240_h16x4_8bit", op="archive", layers=4, slots=240, heads=16, rows=70, bits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "verify", "logprobs", "logprobs", "archive"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    H = rng.choice([1, 2, 4, 8, 16])
    HV = H * rng.choice([1, 1, 2, 4]) if H <= 8 else H * rng.choice([1, 2])
    gate, norm = rng.choice(["raw", "given", "fixed"]), rng.random() < 0.6
    if op == "prefill":
        n = _log_int(rng, 1, 24)
        top = max(2, min(8192, 16384 // n))
        lengths = [rng.choice([0, 1]) if rng.random() < 0.1 else _log_int(rng, 1, top) for _ in range(n)]
        if sum(lengths) == 0:
            lengths[0] = 1
        HV = HV if HV <= 16 else H
        return dict(op=op, lengths=",".join(map(str, lengths)), H=H, HV=HV, slots=n + rng.randint(0, 40),
                    pad=rng.choice([0, rng.randint(1, 500)]), dtype=dtype, gate=gate, norm=norm)
    if op == "decode":
        B = _log_int(rng, 1, 48)
        return dict(op=op, B=B, H=H, HV=HV, slots=B + rng.randint(0, 100), dtype=dtype, gate=gate, norm=norm)
    if op == "verify":
        B, T = _log_int(rng, 1, 24), rng.randint(1, 10)
        return dict(op=op, B=B, T=T, tree=rng.random() < 0.5, H=H, HV=HV if HV <= 16 else H, slots=B + rng.randint(0, 100),
                    dtype=dtype, gate=gate, norm=norm)
    if op == "logprobs":
        return dict(op=op, rows=_log_int(rng, 1, 288), vocab=_log_int(rng, 2, 131072), top=rng.choice([0, 1, 5, 20, 32]),
                    pad=rng.choice([0, 0, rng.randint(1, 64)]), masked=rng.random() < 0.3, idle=rng.random() < 0.3,
                    dtype=rng.choice(["f32", "bf16", "f16"]))
    slots = _log_int(rng, 2, 240)
    return dict(op=op, layers=rng.randint(1, 3), slots=slots, heads=rng.choice([1, 4, 16]), rows=rng.randint(1, max(1, slots // 3)),
                bits=rng.choice([8, 4]))


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def work(case):
    op = case["op"]
    if op == "archive":
        # stored: a page read, its codes and scales written; read back the other way
        n = case["rows"] * case["layers"] * case["heads"] * V * K
        bits = case["bits"]
        return {"bytes": 2.0 * n * (4 + bits / 8 + 4 / GROUP[bits]), "flops": 4.0 * n}
    if op == "logprobs":
        es = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * es + 12.0 + 8 * case["top"]), "flops": 5.0 * case["rows"] * case["vocab"]}
    H, HV = case["H"], case["HV"]
    gate = {"raw": 2, "given": 4, "fixed": 0}[case["gate"]] * HV
    token = 2 * H * K * 2 + 2 * HV * V * 2 + gate
    state = HV * V * K * 4
    if op == "prefill":
        ls = _lengths(case)
        T, n = sum(ls), len(ls)
        # per token and value head: q S and k v^T, and half of a 64-token square twice
        return {"bytes": T * token + 2.0 * n * state, "flops": T * HV * (4.0 * K * V + 2.0 * (CHUNK / 2) * (K + V))}
    if op == "decode":
        return {"bytes": case["B"] * (token + 2.0 * state), "flops": case["B"] * HV * 5.0 * K * V}
    B, T = case["B"], case["T"]
    return {"bytes": B * (T * token + (1.0 + T) * state), "flops": B * T * HV * 5.0 * K * V}


# ---------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _gate_inputs(g, case, rows, real):
    """Gate inputs of `rows` rows; those past `real` are bucket padding (never
    to be read).  Rates exp(A_log) of 1 to 16 and softplus(dt_bias) of 0.001 to
    0.1, the usual start of layers whose decay follows the token; rates of 1/2
    down to 1/256 over the heads where it is fixed."""
    HV = case["HV"]
    if case["gate"] == "fixed":
        return -8 * math.log(2) / HV * torch.arange(1, HV + 1, device="cuda", dtype=torch.float32), None, None
    A_log = torch.log(torch.empty(HV, device="cuda").uniform_(1, 16, generator=g))
    step = torch.exp(torch.empty(HV, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=g))
    dt_bias = step + torch.log(-torch.expm1(-step))
    a = torch.randn(rows, HV, device="cuda", generator=g)
    if case["gate"] == "given":
        a = -torch.exp(A_log) * torch.log1p(torch.exp(a + dt_bias))
        A_log = dt_bias = None
    else:
        a = a.to(TYPES[case["dtype"]])
    a[real:] = float("nan")
    return A_log, dt_bias, a


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "prefill":
        ls = _lengths(case)
        T, n, H, HV, dt = sum(ls), len(ls), case["H"], case["HV"], TYPES[case["dtype"]]
        for name, heads in (("q", H), ("k", H), ("v", HV)):
            s[name] = torch.randn(T, heads, K, device="cuda", generator=g).to(dt)
        s["A_log"], s["dt_bias"], s["a"] = _gate_inputs(g, case, T + case["pad"], T)
        s["pool"] = torch.randn(case["slots"], HV, V, K, device="cuda", generator=g) * 0.02
        s["idx"] = torch.randperm(case["slots"], device="cuda", generator=g)[:n].int()
        s["cu"] = torch.tensor([0] + torch.tensor(ls).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        s["n"], s["o"] = n, torch.empty(T, HV, V, dtype=dt, device="cuda")
    elif op in ("decode", "verify"):
        B, T, H, HV, dt = case["B"], case.get("T", 1), case["H"], case["HV"], TYPES[case["dtype"]]
        s["qkv"] = torch.randn(B * T, (2 * H + HV) * K, device="cuda", generator=g).to(dt)
        s["A_log"], s["dt_bias"], s["a"] = _gate_inputs(g, case, B * T, B * T)
        s["pool"] = torch.randn(case["slots"], HV, V, K, device="cuda", generator=g) * 0.02
        s["idx"] = torch.randperm(case["slots"], device="cuda", generator=g)[:B].int()
        s["parent"] = None
        if case.get("tree"):
            i = torch.arange(T, device="cuda")
            u = torch.rand(B, T, device="cuda", generator=g)
            s["parent"] = torch.minimum((u * i).floor().long(), (i - 1).clamp(min=0)).int()
            s["parent"][:, 0] = -1
        if op == "decode":
            s["o"] = torch.empty(B, HV, V, dtype=dt, device="cuda")
        else:
            s["o"] = torch.empty(B, T, HV, V, dtype=dt, device="cuda")
            s["snapshots"] = torch.empty(B, T, HV, V, K, device="cuda")
    elif op == "logprobs":
        # logits of a trained model's kind, rows apart by more than their length where the head is padded
        rows, W, top = case["rows"], case["vocab"], case["top"]
        whole = torch.randn(rows, W + case["pad"], device="cuda", generator=g) * 2.5
        s["logits"] = whole.to(TYPES[case["dtype"]])[:, :W]
        tokens = torch.randint(0, W, (rows,), device="cuda", generator=g)
        likely = s["logits"].argmax(-1)
        tokens = torch.where(torch.rand(rows, device="cuda", generator=g) < 0.5, likely, tokens)
        if case["masked"]:  # a grammar: a few of the entries may follow, in the last row just one
            keep = torch.rand(rows, W, device="cuda", generator=g) < 0.05
            keep[-1] = False
            keep[torch.arange(rows, device="cuda"), tokens] = True
            s["logits"].masked_fill_(~keep, -torch.inf)
        if case["idle"]:  # rows that nothing is asked of
            tokens = torch.where(torch.rand(rows, device="cuda", generator=g) < 0.1, -1, tokens)
        s["tokens"] = tokens.int()
        s["logprobs"] = torch.empty(rows, device="cuda")
        s["entropy"] = torch.empty(rows, device="cuda")
        s["top_tokens"] = torch.empty(rows, top, dtype=torch.int32, device="cuda") if top else None
        s["top_logprobs"] = torch.empty(rows, top, device="cuda") if top else None
    else:
        L, slots, HV, n, bits = case["layers"], case["slots"], case["heads"], case["rows"], case["bits"]
        # states of heads that decay at different rates
        s["pool"] = torch.randn(L, slots, HV, V, K, device="cuda", generator=g)
        s["pool"] *= torch.exp(torch.randn(L, slots, HV, 1, K, device="cuda", generator=g) * 0.5)
        order = torch.randperm(slots, device="cuda", generator=g).int()
        s["src"], s["dst"] = order[:n].clone(), order[slots - n:].clone()
        s["kept"] = torch.randperm(n + 3, device="cuda", generator=g)[:n].int()
        s["codes"] = (torch.zeros(n + 3, L, HV, V, K, dtype=torch.int8, device="cuda") if bits == 8 else
                      torch.zeros(n + 3, L, HV, V, K // 2, dtype=torch.uint8, device="cuda"))
        s["scales"] = torch.zeros(n + 3, L, HV, V, K // GROUP[bits], device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass


def run(s):
    return {"prefill": _prefill, "decode": _decode, "verify": _verify, "logprobs": _logprobs, "archive": _archive}[s["case"]["op"]](s)


def _library(s):
    from linear_attention_serving_gated_gb300 import kda

    c = s["case"]
    if "H" not in c:
        return kda, None, None
    d = kda.dims(c["H"], HV=c["HV"], dtype=kda.KDA_DTYPE_F16 if c["dtype"] == "f16" else kda.KDA_DTYPE_BF16)
    return kda, d, kda.ScalarGate(A_log=s["A_log"], dt_bias=s["dt_bias"], use_qk_l2norm=c["norm"])


def _prefill(s):
    if own:
        kda, d, gate = _library(s)
        kda.kda_lin_prefill(d, gate, s["q"], s["k"], s["v"], s["a"], s["pool"], s["idx"], s["cu"], s["n"], s["o"])
    else:
        _plain_prefill(s)
    return {"o": s["o"], "pool": s["pool"]}


def _decode(s):
    if own:
        kda, d, gate = _library(s)
        kda.kda_lin_decode_packed(d, gate, s["qkv"], s["a"], s["pool"], s["idx"], s["o"])
    else:
        idx = s["idx"].long()
        q, k, v, decay = _plain_packed(s, s["case"]["B"], 1)
        S, o = _plain_token(s["pool"][idx], q[:, 0], k[:, 0], v[:, 0], decay[:, 0])
        s["pool"][idx] = S
        s["o"].copy_(o)
    return {"o": s["o"], "pool": s["pool"]}


def _verify(s):
    c = s["case"]
    if own:
        kda, d, gate = _library(s)
        if s["parent"] is None:
            kda.kda_lin_verify_chain(d, gate, s["qkv"], s["a"], c["B"], c["T"], s["pool"], s["idx"], s["o"], s["snapshots"])
        else:
            kda.kda_lin_verify_tree(d, gate, s["qkv"], s["a"], c["B"], c["T"], s["parent"], s["pool"], s["idx"], s["o"], s["snapshots"])
    else:
        q, k, v, decay = _plain_packed(s, c["B"], c["T"])
        root = s["pool"][s["idx"].long()]
        at = torch.arange(c["B"], device="cuda")
        S = root
        for t in range(c["T"]):
            if s["parent"] is not None and t > 0:
                p = s["parent"][:, t].long()
                S = torch.where((p < 0)[:, None, None, None], root, s["snapshots"][at, p.clamp(min=0)])
            S, o = _plain_token(S, q[:, t], k[:, t], v[:, t], decay[:, t])
            s["snapshots"][:, t] = S
            s["o"][:, t] = o
    return {"o": s["o"], "snapshots": s["snapshots"]}


def _logprobs(s):
    if own:
        kda, _, _ = _library(s)
        kda.kda_token_logprobs(s["logits"], s["tokens"], s["logprobs"], entropy=s["entropy"], top_tokens=s["top_tokens"],
                               top_logprobs=s["top_logprobs"])
    else:
        _plain_logprobs(s)
    out = {"logprobs": s["logprobs"], "entropy": s["entropy"]}
    if s["top_tokens"] is not None:
        out.update(top_tokens=s["top_tokens"], top_logprobs=s["top_logprobs"])
    return out


def _archive(s):
    """Pages into the archive, and other pages of the pool filled from it."""
    if own:
        kda, _, _ = _library(s)
        kda.kda_pool_store(s["pool"], s["codes"], s["scales"], s["src"], s["kept"])
        kda.kda_pool_load(s["codes"], s["scales"], s["pool"], s["kept"], s["dst"])
    else:
        bits, kept = s["case"]["bits"], s["kept"].long()
        x = s["pool"][:, s["src"].long()].transpose(0, 1).unflatten(-1, (-1, GROUP[bits]))
        scale = x.abs().amax(-1)
        scale = scale / torch.full_like(scale, TOP[bits])
        # the code is the nearest whole number, ties to even: quotients next to a half need 64 bits
        code = torch.where(scale[..., None] > 0, x.double() / scale.double()[..., None], 0).round().clamp(-TOP[bits], TOP[bits])
        code = code.flatten(-2).to(torch.int8)
        if bits == 4:
            s["codes"][kept] = ((code[..., 0::2] & 15) | (code[..., 1::2] << 4)).view(torch.uint8)
        else:
            s["codes"][kept] = code
        s["scales"][kept] = scale
        code = s["codes"][kept]
        if bits == 4:
            code = code.view(torch.int8)
            code = torch.stack([(code << 4) >> 4, code >> 4], -1).flatten(-2)
        value = code.float().unflatten(-1, (-1, GROUP[bits])) * s["scales"][kept][..., None]
        s["pool"][:, s["dst"].long()] = value.flatten(-2).transpose(0, 1)
    return {"pool": s["pool"], "scales": s["scales"]}


# ---------------------------------------------------------------------------
# plain forms


def _norm(s, x):
    x = x.float()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) if s["case"]["norm"] else x


def _plain_gate(s, rows):
    if s["a"] is None:
        return (-torch.exp(s["A_log"])).expand(rows, -1)
    a = s["a"][:rows].float()
    if s["A_log"] is not None:
        x = a + s["dt_bias"]
        # softplus, from the side that does not overflow
        a = -torch.exp(s["A_log"]) * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))
    return a


def _plain_packed(s, B, T):
    c = s["case"]
    H, HV = c["H"], c["HV"]
    q, k, v = s["qkv"].view(B, T, -1).split([H * K, H * K, HV * V], -1)
    rep = lambda y: _norm(s, y.reshape(B, T, H, K)).repeat_interleave(HV // H, 2)  # noqa: E731
    return rep(q), rep(k), v.reshape(B, T, HV, V).float(), torch.exp(_plain_gate(s, B * T)).view(B, T, HV)


def _plain_token(S, q, k, v, decay):
    """One token; S [.., HV, V, K]."""
    S = S * decay[..., None, None] + v[..., :, None] * k[..., None, :]
    return S, K ** -0.5 * (S * q[..., None, :]).sum(-1)


def _plain_prefill(s):
    """Chunks of 64 tokens.  With c_i the log-decay summed up to token i inside
    a chunk and S the state before it:
        O = scale (e^c Q S + [e^(c_i - c_j) q_i.k_j, j <= i] V)
        S' = e^c_last S + sum_j e^(c_last - c_j) k_j v_j^T"""
    c = s["case"]
    H, HV, n = c["H"], c["HV"], s["n"]
    ls = _lengths(c)
    idx = s["idx"].long()
    S = s["pool"][idx].transpose(-1, -2).contiguous()  # [n, HV, K, V]
    chunks = -(-max(ls) // CHUNK)
    T, L = sum(ls), chunks * CHUNK
    # every sequence padded with tokens that change nothing: k = v = g = 0
    cu = s["cu"].long()
    at = cu[:-1, None] + torch.arange(L, device="cuda")
    real = torch.arange(L, device="cuda") < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(real, at, 0)
    lay = lambda x, heads: (torch.where(real[..., None, None], x[at], 0).repeat_interleave(HV // heads, 2)  # noqa: E731
                            .view(n, chunks, CHUNK, HV, -1).permute(1, 0, 3, 2, 4))
    q, k, v = lay(_norm(s, s["q"]), H), lay(_norm(s, s["k"]), H), lay(s["v"].float(), HV)
    g = lay(_plain_gate(s, T)[..., None], HV).squeeze(-1)
    cum = g.double().cumsum(-1)  # sums over 64 tokens, whose differences count
    i = torch.arange(CHUNK, device="cuda")
    low = i[:, None] >= i
    o = torch.empty(chunks, n, HV, CHUNK, V, device="cuda")
    for j in range(chunks):
        cj = cum[j]
        D = torch.exp(torch.where(low, cj[..., :, None] - cj[..., None, :], -torch.inf)).float()
        o[j] = K ** -0.5 * (torch.exp(cj).float()[..., None] * (q[j] @ S) + (D * (q[j] @ k[j].transpose(-1, -2))) @ v[j])
        left = torch.exp(cj[..., -1:] - cj).float()
        S = torch.exp(cj[..., -1, None, None]).float() * S + (left[..., None] * k[j]).transpose(-1, -2) @ v[j]
    s["pool"][idx] = S.transpose(-1, -2)
    o = o.permute(1, 0, 3, 2, 4).reshape(n, L, HV, V)
    s["o"].copy_(o[real])


def _plain_logprobs(s):
    """With m a row's largest logit and z = sum exp(x - m):
        log p = x - m - log z,   entropy = log z - sum (x - m) exp(x - m) / z
    Alternatives by falling logit, the lowest token first among equals; masked
    ones (-inf) are none, places left over hold -1 and -inf.  A row whose token
    is -1 gives zeros, and -1 as its alternatives."""
    x, tokens = s["logits"].float(), s["tokens"].long()
    live = tokens >= 0
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    z = e.double().sum(-1)
    log_z = torch.log(z)
    at = torch.arange(len(tokens), device="cuda")
    s["logprobs"].copy_(torch.where(live, d[at, tokens.clamp(min=0)].double() - log_z, 0))
    mean = torch.where(e > 0, d * e, 0).double().sum(-1) / z
    s["entropy"].copy_(torch.where(live, log_z - mean, 0))
    top = s["case"]["top"]
    if top:
        best, token = torch.sort(x, dim=-1, descending=True, stable=True)
        n = min(top, x.shape[1])
        best, token = best[:, :n], torch.where(best[:, :n] > -torch.inf, token[:, :n], -1)
        s["top_tokens"].fill_(-1)
        s["top_logprobs"].fill_(-torch.inf)
        s["top_tokens"][:, :n] = torch.where(live[:, None], token, -1)
        s["top_logprobs"][:, :n] = (best - m).double() - log_z[:, None]
        s["top_logprobs"][~live] = 0


# ---------------------------------------------------------------------------
# in 64 bits, token by token from the rule


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    f64 = torch.float64
    if op == "archive":
        bits = case["bits"]
        top, group = TOP[bits], GROUP[bits]
        pool, scales = s["pool"].to(f64), s["scales"].to(f64)
        for src, kept, dst in zip(s["src"].tolist(), s["kept"].tolist(), s["dst"].tolist()):
            x = s["pool"][:, src].to(f64).reshape(-1, group)
            unit = (x.abs().max(-1).values / top).float().to(f64)  # a scale is an FP32 number
            code = torch.round(x / unit.clamp(min=1e-300)[:, None]).clamp(-top, top)
            scales[kept] = unit.view(scales[kept].shape)
            pool[:, dst] = (code * unit[:, None]).view(pool[:, dst].shape)
        return {"pool": pool, "scales": scales}
    if op == "logprobs":
        out = {"logprobs": torch.zeros(case["rows"], dtype=f64, device="cuda"), "entropy": torch.zeros(case["rows"], dtype=f64, device="cuda")}
        top = case["top"]
        if top:
            out["top_tokens"] = torch.full((case["rows"], top), -1, dtype=torch.int32, device="cuda")
            out["top_logprobs"] = torch.zeros(case["rows"], top, dtype=f64, device="cuda")
        for r, t in enumerate(s["tokens"].tolist()):
            if t < 0:
                continue
            x = s["logits"][r].to(f64)
            lp = x - torch.logsumexp(x, 0)
            out["logprobs"][r] = lp[t]
            there = lp[lp > -torch.inf]
            out["entropy"][r] = -(there.exp() * there).sum()
            if top:
                order = torch.argsort(x, descending=True, stable=True)[:min(top, len(there))]
                out["top_logprobs"][r] = -torch.inf
                out["top_logprobs"][r, :len(order)] = lp[order]
                out["top_tokens"][r, :len(order)] = order.int()
        return out
    H, HV = case["H"], case["HV"]
    if case["gate"] == "fixed":
        rows = s["q"].shape[0] if op == "prefill" else s["qkv"].shape[0]
        alpha = (-s["A_log"].to(f64).exp()).exp().expand(rows, HV).contiguous()
    elif case["gate"] == "given":
        alpha = s["a"].to(f64).exp()
    else:
        alpha = (-s["A_log"].to(f64).exp() * torch.nn.functional.softplus(s["a"].to(f64) + s["dt_bias"].to(f64), threshold=700)).exp()
    unit = lambda x: x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt() if case["norm"] else x  # noqa: E731
    pool = s["pool"].to(f64)

    def step(S, q, k, v, al):
        """S [m, HV, K, V] -> (S_t, o_t)."""
        q, k = (unit(x.to(f64)).repeat_interleave(HV // H, 1) for x in (q, k))
        S = al[..., None, None] * S + k[..., :, None] * v.to(f64)[..., None, :]
        return S, K ** -0.5 * torch.einsum("nhkv,nhk->nhv", S, q)

    if op == "prefill":
        ls = _lengths(case)
        if max(ls) * sum(1 for x in ls if x) > 120000:
            return None
        order = sorted(range(len(ls)), key=lambda j: -ls[j])
        first = s["cu"].long()[:-1][order]
        S = pool[s["idx"].long()].transpose(-1, -2).clone()[order]
        o = torch.zeros(sum(ls), HV, V, dtype=f64, device="cuda")
        live = len(ls)
        for t in range(max(ls)):
            while live and ls[order[live - 1]] <= t:
                live -= 1
            row = first[:live] + t
            S[:live], o[row] = step(S[:live], s["q"][row], s["k"][row], s["v"][row], alpha[row])
        pool[s["idx"].long()[order]] = S.transpose(-1, -2)
        return {"o": o, "pool": pool}
    B, T = case["B"], case.get("T", 1)
    x = s["qkv"].view(B, T, -1)
    q, k = x[..., :H * K].reshape(B, T, H, K), x[..., H * K:2 * H * K].reshape(B, T, H, K)
    v = x[..., 2 * H * K:].reshape(B, T, HV, V)
    alpha = alpha.view(B, T, HV)
    root = pool[s["idx"].long()].transpose(-1, -2)
    states, outs = [], []
    for t in range(T):
        if t == 0:
            S = root
        elif s["parent"] is None:
            S = states[-1]
        else:
            S = torch.stack([states[int(p)][r] if p >= 0 else root[r] for r, p in enumerate(s["parent"][:, t].tolist())])
        S, o = step(S, q[:, t], k[:, t], v[:, t], alpha[:, t])
        states.append(S)
        outs.append(o)
    if op == "decode":
        pool[s["idx"].long()] = states[0].transpose(-1, -2)
        return {"o": outs[0], "pool": pool}
    return {"o": torch.stack(outs, 1), "snapshots": torch.stack(states, 1).transpose(-1, -2)}
