"""Cases and plain forms of the serving operators beside the KDA phases: the
gated delta rule with one decay per head (chunked prefill, packed decode,
chain/tree verify), the verification of drafted tokens against the target's
probabilities, and the pages of a state pool (free, compact, fork).

`own` selects what `run` computes with: False, elementary torch operations;
True, the library's entry points.

The rule, per value head, S a K x V state, one log-decay g_t per token:
    S_t = (I - beta_t k_t k_t^T) exp(g_t) S_{t-1} + beta_t k_t v_t^T
    o_t = scale S_t^T q_t
    g_t = -exp(A_log) softplus(a_t + dt_bias), or given;  beta_t = sigmoid(b_t)
    q, k divided by sqrt(sum x^2 + 1e-6)
"""
import math

import torch

own = False

K = V = 128
CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one short prompt of a small model: latency counts
        dict(name="prefill_1x128_h4", op="prefill", lengths="128", H=4, HV=4, slots=4, pad=0, dtype="bf16", given=False),
        # one prompt of the framework's headline length and heads
        dict(name="prefill_1x4096_h16", op="prefill", lengths="4096", H=16, HV=16, slots=16, pad=0, dtype="bf16", given=False),
        # a scheduler's step over a ragged batch padded to a 32768-row bucket
        dict(name="prefill_varlen8_h16", op="prefill", lengths="1,8087,517,2048,1290,3331,64,1642", H=16, HV=16, slots=240,
             pad=32768 - 16980, dtype="bf16", given=False),
        # grouped value heads, FP16 tokens, log-decays given in FP32, odd lengths
        dict(name="prefill_ragged_f16_h8_hv16", op="prefill", lengths="1000,333,77,2001", H=8, HV=16, slots=16, pad=5,
             dtype="f16", given=True),
        # one user generating: the smallest decode step
        dict(name="decode_1_h16", op="decode", B=1, H=16, HV=16, slots=240, dtype="bf16", given=False),
        # a full decode batch with grouped value heads
        dict(name="decode_48_h16_hv32", op="decode", B=48, H=16, HV=32, slots=240, dtype="bf16", given=False),
        # speculative verify of six tokens for sixteen requests, state snapshots kept
        dict(name="verify_16x6_h16", op="verify", B=16, T=6, tree=False, H=16, HV=16, slots=240, dtype="bf16", given=False),
        # one request's drafts against a 32000-token vocabulary
        dict(name="accept_1x6_v32000", op="accept", B=1, T=6, tree=False, vocab=32000, draft=True, ragged=False, dtype="f32"),
        # a full batch of drafts against a large vocabulary
        dict(name="accept_48x6_v131072", op="accept", B=48, T=6, tree=False, vocab=131072, draft=True, ragged=False, dtype="f32"),
        # draft trees proposed without probabilities, odd vocabulary, 16-bit probabilities
        dict(name="accept_tree_16x6_v50257", op="accept", B=16, T=6, tree=True, vocab=50257, draft=False, ragged=True, dtype="bf16"),
        # a scheduler between two steps of a few requests: one finishes, its page goes to a fork of another
        dict(name="pages_6_of_16_h4", op="pages", layers=1, slots=16, heads=4, rows=6, churn=1),
        # the same for a full pool and several layers: a third of the requests finish
        dict(name="pages_210_of_240_h16x4", op="pages", layers=4, slots=240, heads=16, rows=210, churn=70),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "verify", "accept", "accept", "pages"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    H = rng.choice([1, 2, 4, 8, 16])
    HV = H * rng.choice([1, 1, 2, 4]) if H <= 8 else H * rng.choice([1, 2])
    given = rng.random() < 0.3
    if op == "prefill":
        n = _log_int(rng, 1, 24)
        top = max(2, min(8192, 16384 // n))
        lengths = [rng.choice([0, 1]) if rng.random() < 0.1 else _log_int(rng, 1, top) for _ in range(n)]
        if sum(lengths) == 0:
            lengths[0] = 1
        HV = min(HV, 16) if HV % H == 0 and min(HV, 16) % H == 0 else H
        return dict(op=op, lengths=",".join(map(str, lengths)), H=H, HV=HV, slots=n + rng.randint(0, 40),
                    pad=rng.choice([0, rng.randint(1, 500)]), dtype=dtype, given=given)
    if op == "decode":
        B = _log_int(rng, 1, 48)
        return dict(op=op, B=B, H=H, HV=HV, slots=B + rng.randint(0, 100), dtype=dtype, given=given)
    if op == "verify":
        B, T = _log_int(rng, 1, 24), rng.randint(1, 10)
        return dict(op=op, B=B, T=T, tree=rng.random() < 0.5, H=H, HV=min(HV, 16) if H <= 16 and 16 % H == 0 else H,
                    slots=B + rng.randint(0, 100), dtype=dtype, given=given)
    if op == "accept":
        tree = rng.random() < 0.4
        return dict(op=op, B=_log_int(rng, 1, 48), T=rng.randint(1, 16 if tree else 8), tree=tree, vocab=_log_int(rng, 2, 131072),
                    draft=not tree and rng.random() < 0.7, ragged=rng.random() < 0.4, dtype=rng.choice(["f32", "f32", "bf16", "f16"]))
    slots = _log_int(rng, 2, 240)
    rows = rng.randint(2, slots)
    return dict(op="pages", layers=rng.randint(1, 3), slots=slots, heads=rng.choice([1, 4, 16]), rows=rows,
                churn=rng.randint(1, max(1, rows // 3)))


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def work(case):
    op = case["op"]
    if op == "pages":
        # every page that moves or is forked is read once and written once.  The
        # rows that go are spread over the table, so the holes below the new
        # top number about churn (rows - churn) / rows; each takes one page
        page = case["heads"] * V * K * 4 * case["layers"]
        rows, churn = case["rows"], case["churn"]
        moves = churn * (rows - churn) / rows
        return {"bytes": 2.0 * page * (moves + churn), "flops": 0}
    if op == "accept":
        es = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["B"] * (case["vocab"] * es * (2 if case["draft"] else 1) + case["T"] * 12.0), "flops": 3.0 * case["B"] * case["vocab"]}
    H, HV = case["H"], case["HV"]
    gate = HV * (4 if case["given"] else 2) + HV * 2
    token = 2 * H * K * 2 + 2 * HV * V * 2 + gate
    state = HV * V * K * 4
    if op == "prefill":
        ls = _lengths(case)
        T, n = sum(ls), len(ls)
        # per token and head: q S, k S, k v^T updates, and the 64-token triangles
        flops = T * HV * (6.0 * K * V + 2.0 * (CHUNK / 2) * (2 * K + 2 * V))
        return {"bytes": T * token + 2.0 * n * state, "flops": flops}
    if op == "decode":
        return {"bytes": case["B"] * (token + 2.0 * state), "flops": case["B"] * HV * 7.0 * K * V}
    B, T = case["B"], case["T"]
    return {"bytes": B * (T * token + (1.0 + T) * state), "flops": B * T * HV * 7.0 * K * V}


# ---------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _gate_inputs(g, case, rows, real):
    """Gate inputs of `rows` rows; those past `real` are bucket padding (never
    to be read).  Decay rates: exp(A_log) in 1..16, softplus(dt_bias) in
    0.001..0.1, the usual start of such layers."""
    HV, dt = case["HV"], TYPES[case["dtype"]]
    A_log = torch.log(torch.empty(HV, device="cuda").uniform_(1, 16, generator=g))
    step = torch.exp(torch.empty(HV, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=g))
    dt_bias = step + torch.log(-torch.expm1(-step))
    a = torch.randn(rows, HV, device="cuda", generator=g)
    b = torch.randn(rows, HV, device="cuda", generator=g)
    if case["given"]:
        a = -torch.exp(A_log) * torch.log1p(torch.exp(a + dt_bias))
        A_log = dt_bias = None
    else:
        a = a.to(dt)
    b = b.to(dt)
    a[real:] = float("nan")
    b[real:] = 3e4
    return A_log, dt_bias, a, b


def _chain_or_tree(g, B, T, tree):
    if not tree:
        return None
    u = torch.rand(B, T, device="cuda", generator=g)
    i = torch.arange(T, device="cuda")
    parent = torch.minimum((u * i).floor().long(), (i - 1).clamp(min=0))
    parent[:, 0] = -1
    return parent.int()


def _peaked(g, shape, dtype, base=None):
    """Probabilities of a trained model's kind: a softmax over spread logits;
    with `base`, a draft model's, near the target's."""
    logits = torch.randn(shape, device="cuda", generator=g) * 2.5
    if base is not None:
        logits = base + 0.4 * logits
    p = torch.softmax(logits, -1)
    return logits, p.to(TYPES[dtype])


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "prefill":
        ls = _lengths(case)
        T, n, H, HV, dt = sum(ls), len(ls), case["H"], case["HV"], TYPES[case["dtype"]]
        for name, heads in (("q", H), ("k", H), ("v", HV)):
            s[name] = torch.randn(T, heads, K, device="cuda", generator=g).to(dt)
        s["A_log"], s["dt_bias"], s["a"], s["b"] = _gate_inputs(g, case, T + case["pad"], T)
        s["pool"] = torch.randn(case["slots"], HV, V, K, device="cuda", generator=g) * 0.02
        s["idx"] = torch.randperm(case["slots"], device="cuda", generator=g)[:n].int()
        s["cu"] = torch.tensor([0] + torch.tensor(ls).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        s["n"], s["o"] = n, torch.empty(T, HV, V, dtype=dt, device="cuda")
    elif op in ("decode", "verify"):
        B, T, H, HV, dt = case["B"], case.get("T", 1), case["H"], case["HV"], TYPES[case["dtype"]]
        s["qkv"] = torch.randn(B * T, (2 * H + HV) * K, device="cuda", generator=g).to(dt)
        s["A_log"], s["dt_bias"], s["a"], s["b"] = _gate_inputs(g, case, B * T, B * T)
        s["pool"] = torch.randn(case["slots"], HV, V, K, device="cuda", generator=g) * 0.02
        s["idx"] = torch.randperm(case["slots"], device="cuda", generator=g)[:B].int()
        s["parent"] = _chain_or_tree(g, B, T, case.get("tree", False))
        if op == "decode":
            s["o"] = torch.empty(B, HV, V, dtype=dt, device="cuda")
        else:
            s["o"] = torch.empty(B, T, HV, V, dtype=dt, device="cuda")
            s["snapshots"] = torch.empty(B, T, HV, V, K, device="cuda")
    elif op == "accept":
        B, T, W = case["B"], case["T"], case["vocab"]
        logits, s["target"] = _peaked(g, (B, T, W), case["dtype"])
        s["draft"] = None
        tokens = torch.randint(0, W, (B, T), device="cuda", generator=g)
        s["parent"] = _chain_or_tree(g, B, T, case["tree"])
        if T > 1:
            if case["draft"]:
                _, s["draft"] = _peaked(g, (B, T - 1, W), case["dtype"], logits[:, :-1])
                tokens[:, 1:] = torch.multinomial(s["draft"].float().view(-1, W), 1, generator=g).view(B, T - 1)
            else:  # proposed without probabilities: likely tokens of the node they follow
                likely = logits.topk(min(4, W), -1).indices
                up = s["parent"][:, 1:].long() if case["tree"] else torch.arange(T - 1, device="cuda").expand(B, -1)
                pick = torch.randint(0, likely.shape[-1], (B, T - 1, 1), device="cuda", generator=g)
                tokens[:, 1:] = likely.gather(1, up.unsqueeze(-1).expand(-1, -1, likely.shape[-1])).gather(2, pick).squeeze(-1)
        s["tokens"] = tokens.int()
        s["u"] = torch.rand(B, T, device="cuda", generator=g)
        s["lengths"] = torch.randint(0, T + 1, (B,), device="cuda", generator=g).int() if case["ragged"] else None
        s["accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["next"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["path"] = torch.empty(B, T, dtype=torch.int32, device="cuda")
    else:
        slots, rows = case["slots"], case["rows"]
        s["pool"] = torch.randn(case["layers"], slots, case["heads"], V, K, device="cuda", generator=g)
        s["table"] = torch.randperm(slots, device="cuda", generator=g)[:rows].int()
        s["used"] = torch.zeros(slots, dtype=torch.uint8, device="cuda")
        s["used"][s["table"].long()] = 1
        order = torch.randperm(rows, device="cuda", generator=g)
        churn = case["churn"]
        s["gone"] = order[:churn].sort().values.int()  # table rows of the requests that finish
        stay = order[churn:]
        s["forked"] = stay[torch.randint(0, len(stay), (churn,), device="cuda", generator=g)].int()  # whom their rows continue
        s["count"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass


def run(s):
    op = s["case"]["op"]
    if op == "prefill":
        return _prefill(s)
    if op == "decode":
        return _decode(s)
    if op == "verify":
        return _verify(s)
    if op == "accept":
        return _accept(s)
    return _pages(s)


def _library(s):
    from linear_attention_serving_gated_gb300 import kda

    c = s["case"]
    if "H" not in c:
        return kda, None, None
    d = kda.dims(c["H"], HV=c["HV"], dtype=kda.KDA_DTYPE_F16 if c["dtype"] == "f16" else kda.KDA_DTYPE_BF16)
    return kda, d, kda.ScalarGate(A_log=s["A_log"], dt_bias=s["dt_bias"])


def _prefill(s):
    if own:
        kda, d, gate = _library(s)
        kda.kda_gdn_prefill(d, gate, s["q"], s["k"], s["v"], s["a"], s["b"], s["pool"], s["idx"], s["cu"], s["n"], s["o"])
    else:
        _plain_prefill(s)
    return {"o": s["o"], "pool": s["pool"]}


def _decode(s):
    if own:
        kda, d, gate = _library(s)
        kda.kda_gdn_decode_packed(d, gate, s["qkv"], s["a"], s["b"], s["pool"], s["idx"], s["o"])
    else:
        c = s["case"]
        idx = s["idx"].long()
        q, k, v, decay, beta = _plain_packed(s, c["B"], 1)
        S, o = _plain_token(s["pool"][idx], q[:, 0], k[:, 0], v[:, 0], decay[:, 0], beta[:, 0])
        s["pool"][idx] = S
        s["o"].copy_(o)
    return {"o": s["o"], "pool": s["pool"]}


def _verify(s):
    c = s["case"]
    if own:
        kda, d, gate = _library(s)
        if s["parent"] is None:
            kda.kda_gdn_verify_chain(d, gate, s["qkv"], s["a"], s["b"], c["B"], c["T"], s["pool"], s["idx"], s["o"], s["snapshots"])
        else:
            kda.kda_gdn_verify_tree(d, gate, s["qkv"], s["a"], s["b"], c["B"], c["T"], s["parent"], s["pool"], s["idx"], s["o"],
                                    s["snapshots"])
    else:
        q, k, v, decay, beta = _plain_packed(s, c["B"], c["T"])
        root = s["pool"][s["idx"].long()]
        at = torch.arange(c["B"], device="cuda")
        S = root
        for t in range(c["T"]):
            if s["parent"] is not None and t > 0:
                p = s["parent"][:, t].long()
                S = torch.where((p < 0)[:, None, None, None], root, s["snapshots"][at, p.clamp(min=0)])
            S, o = _plain_token(S, q[:, t], k[:, t], v[:, t], decay[:, t], beta[:, t])
            s["snapshots"][:, t] = S
            s["o"][:, t] = o
    return {"o": s["o"], "snapshots": s["snapshots"]}


def _accept(s):
    if own:
        kda, _, _ = _library(s)
        if s["parent"] is None:
            kda.kda_accept_chain(s["target"], s["draft"], s["tokens"], s["u"], s["accepted"], s["next"], lengths=s["lengths"])
        else:
            kda.kda_accept_tree(s["target"], s["tokens"], s["parent"], s["u"], s["accepted"], s["path"], s["next"], lengths=s["lengths"])
    elif s["parent"] is None:
        _plain_accept_chain(s)
    else:
        _plain_accept_tree(s)
    return {"accepted": s["accepted"], "next": s["next"]} if s["parent"] is None else {"accepted": s["accepted"], "next": s["next"], "path": s["path"]}


def _pages(s):
    """Between two steps: the pages of the finished requests are freed, the
    pool is compacted, and the rows that became free continue from forks of
    other requests' states."""
    pool, used, table = s["pool"], s["used"], s["table"]
    if own:
        kda, _, _ = _library(s)
        kda.kda_pool_free(used, table, s["gone"])
        kda.kda_pool_compact(pool, used, table, s["count"])
        kda.kda_pool_fork(pool, used, table, s["forked"], s["gone"])
    else:
        gone = s["gone"].long()
        used[table[gone].long()] = 0
        table[gone] = -1
        # the k-th lowest hole below the new top takes the k-th lowest page above it
        slot = torch.arange(used.numel(), device="cuda")
        total = used.sum()
        s["count"].copy_(total.view(1))
        hole = ((used == 0) & (slot < total)).nonzero().view(-1)
        above = ((used == 1) & (slot >= total)).nonzero().view(-1)
        pool[:, hole] = pool[:, above]
        to = slot.clone()
        to[above] = hole
        table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
        used.copy_(slot < total)
        # forks take the lowest free pages in order
        free = (used == 0).nonzero().view(-1)[:len(gone)]
        pool[:, free] = pool[:, table[s["forked"].long()].long()]
        used[free] = 1
        table[gone] = free.int()
    return {"pool": pool, "used": used, "table": table, "count": s["count"]}


# ---------------------------------------------------------------------------
# plain forms


def _norm(x):
    x = x.float()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _plain_gate(s, rows):
    a, b = s["a"][:rows].float(), s["b"][:rows].float()
    if s["A_log"] is not None:
        x = a + s["dt_bias"]
        # softplus, from the side that does not overflow
        a = -torch.exp(s["A_log"]) * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))
    return a, 1 / (1 + torch.exp(-b))


def _plain_packed(s, B, T):
    c = s["case"]
    H, HV = c["H"], c["HV"]
    x = s["qkv"].view(B, T, -1)
    q, k, v = x.split([H * K, H * K, HV * V], -1)
    rep = lambda y: _norm(y.reshape(B, T, H, K)).repeat_interleave(HV // H, 2)  # noqa: E731
    g, beta = _plain_gate(s, B * T)
    return rep(q), rep(k), v.reshape(B, T, HV, V).float(), torch.exp(g).view(B, T, HV), beta.view(B, T, HV)


def _plain_token(S, q, k, v, decay, beta):
    """One token; S [.., HV, V, K]."""
    S = S * decay[..., None, None]
    u = beta[..., None] * (v - (S * k[..., None, :]).sum(-1))
    S = S + u[..., :, None] * k[..., None, :]
    return S, K ** -0.5 * (S * q[..., None, :]).sum(-1)


def _plain_prefill(s):
    """Chunks of 64 tokens.  With c_i the log-decay summed up to token i inside
    a chunk and S the state before it:
        A_ij = beta_i e^(c_i - c_j) k_i.k_j (j < i),  (I + A) D = beta (V - e^c K S)
        O = scale (e^c Q S + [e^(c_i - c_j) q_i.k_j, j <= i] D)
        S' = e^c_last S + sum_j e^(c_last - c_j) k_j D_j^T"""
    c = s["case"]
    H, HV, n = c["H"], c["HV"], s["n"]
    ls = _lengths(c)
    idx = s["idx"].long()
    S = s["pool"][idx].transpose(-1, -2).contiguous()  # [n, HV, K, V]
    chunks = -(-max(ls) // CHUNK)
    if chunks == 0:
        return
    T, L = sum(ls), chunks * CHUNK
    # every sequence padded with tokens that change nothing: k = v = beta = g = 0
    cu = s["cu"].long()
    at = cu[:-1, None] + torch.arange(L, device="cuda")
    real = torch.arange(L, device="cuda") < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(real, at, 0)
    lay = lambda x, heads: (torch.where(real[..., None, None], x[at], 0).repeat_interleave(HV // heads, 2)  # noqa: E731
                            .view(n, chunks, CHUNK, HV, -1).permute(1, 0, 3, 2, 4))
    q, k, v = lay(_norm(s["q"]), H), lay(_norm(s["k"]), H), lay(s["v"].float(), HV)
    g, beta = _plain_gate(s, T)
    g, beta = lay(g[..., None], HV).squeeze(-1), lay(beta[..., None], HV).squeeze(-1)
    cum = g.double().cumsum(-1)  # sums over 64 tokens, whose differences count
    i = torch.arange(CHUNK, device="cuda")
    low = i[:, None] >= i
    o = torch.empty(chunks, n, HV, CHUNK, V, device="cuda")
    for j in range(chunks):
        cj = cum[j]
        D = torch.exp(torch.where(low, cj[..., :, None] - cj[..., None, :], -torch.inf)).float()
        up = torch.exp(cj).float()
        kk = k[j] @ k[j].transpose(-1, -2)
        A = beta[j][..., None] * D * kk
        Y = beta[j][..., None] * (v[j] - up[..., None] * (k[j] @ S))
        for t in range(1, CHUNK):
            Y[..., t, :] -= (A[..., t, :t, None] * Y[..., :t, :]).sum(-2)
        o[j] = K ** -0.5 * (up[..., None] * (q[j] @ S) + (D * (q[j] @ k[j].transpose(-1, -2))) @ Y)
        left = torch.exp(cj[..., -1:] - cj).float()
        S = up[..., -1, None, None] * S + (left[..., None] * k[j]).transpose(-1, -2) @ Y
    s["pool"][idx] = S.transpose(-1, -2)
    o = o.permute(1, 0, 3, 2, 4).reshape(n, L, HV, V)
    s["o"].copy_(o[real])


def _weights(p):
    """Probabilities as numbers in 64 bits; NaN, negative and infinite ones
    count as zero."""
    p = p.double()
    return torch.where((p > 0) & (p < torch.inf), p, 0.0)


def _pick(w, u):
    """The lowest token whose running sum passes u times the whole; -1 where
    nothing has weight."""
    cum = w.cumsum(-1)
    over = cum > (u.double() * cum[..., -1])[..., None]
    return torch.where(over.any(-1), over.to(torch.int8).argmax(-1), -1)


def _plain_accept_chain(s):
    """Token i (1..) stands where u_i q(token) < p(token), p the target's row
    i - 1, q the draft's; the first that falls is replaced by a draw from
    max(p - q, 0), and behind the last one a token is drawn from the target."""
    target, draft, tokens, u = s["target"], s["draft"], s["tokens"].long(), s["u"]
    B, T = tokens.shape
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device="cuda")
    at = torch.arange(B, device="cuda")
    stands = torch.ones(B, dtype=torch.bool, device="cuda")
    acc = torch.zeros(B, dtype=torch.long, device="cuda")
    for i in range(1, T):
        p = _weights(target[at, i - 1, tokens[:, i]])
        q = _weights(draft[at, i - 1, tokens[:, i]]) if draft is not None else 1.0
        stands = stands & (u[:, i].double() * q < p) & (i < n)
        acc = acc + stands
    last = acc >= n - 1
    p = _weights(target[at, acc])
    if T > 1:
        row = acc.clamp(max=T - 2)
        if draft is not None:
            q = _weights(draft[at, row])
        else:
            q = torch.zeros_like(p)
            q[at, tokens[at, row + 1]] = torch.inf  # the fallen token has no weight left
        w = torch.where(last[:, None], p, (p - q).clamp(min=0))
        w = torch.where((w > 0).any(-1, keepdim=True), w, p)
    else:
        w = p
    s["accepted"].copy_(torch.where(n > 0, acc, -1))
    s["next"].copy_(torch.where(n > 0, _pick(w, u[:, 0]), -1))


def _plain_accept_tree(s):
    """From the root, the children of the node reached are tried in order of
    their index: child c stands where u_c Z < p(token), Z what the node's
    tried tokens left of 1; where none stands, a token is drawn from what is
    left of the node's row."""
    target, tokens, u, parent = s["target"], s["tokens"].long(), s["u"].double(), s["parent"].long()
    B, T = tokens.shape
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device="cuda")
    at = torch.arange(B, device="cuda")
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    left = torch.ones(B, dtype=torch.float64, device="cuda")
    tried = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    path = torch.full((B, T), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    depth = torch.zeros(B, dtype=torch.long, device="cuda")
    for i in range(1, T):
        mine = (parent[:, i] == cur) & (i < n)
        again = (tried & (tokens == tokens[:, i:i + 1])).any(-1)
        p = torch.where(again, 0.0, _weights(target[at, cur, tokens[:, i]]))
        ok = mine & (u[:, i] * left < p)
        fell = mine & ~ok
        left = torch.where(ok, 1.0, torch.where(fell, left - p, left))
        tried[:, i] = fell
        tried = tried & ~ok[:, None]
        cur = torch.where(ok, i, cur)
        depth = depth + ok
        path[at, depth] = cur
    w = _weights(target[at, cur])
    all_w = w.clone()
    for i in range(1, T):
        w[at[tried[:, i]], tokens[tried[:, i], i]] = 0.0
    w = torch.where((w > 0).any(-1, keepdim=True), w, all_w)
    live = n > 0
    s["accepted"].copy_(torch.where(live, cur, -1))
    s["next"].copy_(torch.where(live, _pick(w, s["u"][:, 0]), -1))
    s["path"].copy_(torch.where(live[:, None], path, -1))


# ---------------------------------------------------------------------------
# in 64 bits, token by token from the rule


def exact(case, seed):
    op = case["op"]
    if op in ("accept", "pages"):
        return None  # whole numbers and copies: equal or wrong
    s = prepare(case, seed)
    H, HV, dt = case["H"], case["HV"], torch.float64
    a, b = s["a"].to(dt), s["b"].to(dt)
    if not case["given"]:
        a = -s["A_log"].to(dt).exp() * torch.nn.functional.softplus(a + s["dt_bias"].to(dt), threshold=700)
    alpha, beta = a.exp(), b.sigmoid()
    unit = lambda x: x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    pool = s["pool"].to(dt)
    scale = K ** -0.5

    def step(S, q, k, v, al, be):
        """S [m, HV, K, V] -> (S_t, o_t)."""
        q, k = unit(q.to(dt)), unit(k.to(dt))
        q, k = (x.repeat_interleave(HV // H, 1) for x in (q, k))
        S = al[..., None, None] * S
        S = S + (be[..., None] * k)[..., :, None] * (v.to(dt) - torch.einsum("nhkv,nhk->nhv", S, k))[..., None, :]
        return S, scale * torch.einsum("nhkv,nhk->nhv", S, q)

    if op == "prefill":
        ls = _lengths(case)
        if max(ls) * sum(1 for x in ls if x) > 120000:
            return None
        start = s["cu"].long()[:-1]
        order = sorted(range(len(ls)), key=lambda j: -ls[j])
        S = pool[s["idx"].long()].transpose(-1, -2).clone()[order]
        o = torch.zeros(sum(ls), HV, V, dtype=dt, device="cuda")
        first = start[order]
        live = len(ls)
        for t in range(max(ls)):
            while live and ls[order[live - 1]] <= t:
                live -= 1
            row = first[:live] + t
            S[:live], o[row] = step(S[:live], s["q"][row], s["k"][row], s["v"][row], alpha[row], beta[row])
        pool[s["idx"].long()[order]] = S.transpose(-1, -2)
        return {"o": o, "pool": pool}
    B, T = case["B"], case.get("T", 1)
    x = s["qkv"].view(B, T, -1)
    q, k = x[..., :H * K].reshape(B, T, H, K), x[..., H * K:2 * H * K].reshape(B, T, H, K)
    v = x[..., 2 * H * K:].reshape(B, T, HV, V)
    alpha, beta = alpha.view(B, T, HV), beta.view(B, T, HV)
    root = pool[s["idx"].long()].transpose(-1, -2)
    states, outs = [], []
    for t in range(T):
        if t == 0:
            S = root
        elif s["parent"] is None:
            S = states[-1]
        else:
            S = torch.stack([states[int(p)][r] if p >= 0 else root[r] for r, p in enumerate(s["parent"][:, t].tolist())])
        S, o = step(S, q[:, t], k[:, t], v[:, t], alpha[:, t], beta[:, t])
        states.append(S)
        outs.append(o)
    if op == "decode":
        pool[s["idx"].long()] = states[0].transpose(-1, -2)
        return {"o": outs[0], "pool": pool}
    return {"o": torch.stack(outs, 1), "snapshots": torch.stack(states, 1).transpose(-1, -2)}
