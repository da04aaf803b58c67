"""FP64 oracles, in numpy and plain Python, of the operators beside the KDA
phases: the gated delta rule with one decay per value head, the verification
of drafted tokens, and the pages of a state pool.  Token by token, request by
request, from the definitions in include/kda.h."""
import numpy as np


def _sigmoid(x):
    return 1 / (1 + np.exp(-x))


def gdn_gate(a, b, A_log=None, dt_bias=None, beta_is_raw=True):
    """Decay factor and beta of every token and value head (arrays [.., HV])."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    if A_log is not None:
        x = a + (0 if dt_bias is None else np.asarray(dt_bias, np.float64))
        a = -np.exp(np.asarray(A_log, np.float64)) * np.logaddexp(0, x)
    return np.exp(a), _sigmoid(b) if beta_is_raw else b


def gdn_step(S, q, k, v, alpha, beta, scale, l2norm=True):
    """One token of all value heads: S [HV,V,K], q,k [H,K], v [HV,V]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    if l2norm:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6) for x in (q, k))
    G = S.shape[0] // q.shape[0]
    q, k = np.repeat(q, G, 0), np.repeat(k, G, 0)
    S = S * alpha[:, None, None]
    u = beta[:, None] * (v - np.einsum("hvk,hk->hv", S, k))
    S = S + u[:, :, None] * k[:, None, :]
    return S, scale * np.einsum("hvk,hk->hv", S, q)


def gdn_sequence(S, q, k, v, alpha, beta, scale, l2norm=True, parents=None):
    """Tokens in order (or a tree): outputs [T,HV,V] and the state behind every
    token [T,HV,V,K]."""
    states, outs = [], []
    for t in range(len(q)):
        p = t - 1 if parents is None else parents[t]
        S_t, o = gdn_step(S if p < 0 else states[p], q[t], k[t], v[t], alpha[t], beta[t], scale, l2norm)
        states.append(S_t)
        outs.append(o)
    return np.array(outs), np.array(states)


def _weights(p):
    p = np.asarray(p, np.float64)
    return np.where((p > 0) & (p < np.inf), p, 0.0)


def draw(w, u):
    """The lowest j whose running sum of w passes u times the whole, -1 where
    nothing has weight."""
    cum = np.cumsum(w)
    if not cum[-1] > 0:
        return -1
    j = int(np.searchsorted(cum, np.float64(u) * cum[-1], side="right"))
    return min(j, int(np.nonzero(w)[0][-1]))


def accept_chain(target, draft, tokens, u, n):
    """One request: target [T,V], draft [T-1,V] or None, n rows."""
    if n <= 0:
        return -1, -1
    V = target.shape[1]
    a = 0
    for i in range(1, n):
        t = tokens[i]
        ok = 0 <= t < V
        p = _weights(target[i - 1, t]) if ok else 0.0
        q = 1.0 if draft is None else _weights(draft[i - 1, t]) if ok else 0.0
        if not np.float64(u[i]) * q < p:
            break
        a = i
    w = p = _weights(target[a])
    if a + 1 < n:
        if draft is not None:
            w = np.maximum(p - _weights(draft[a]), 0)
        else:
            w = p.copy()
            if 0 <= tokens[a + 1] < V:
                w[tokens[a + 1]] = 0
        if not w.any():
            w = p
    return a, draw(w, u[0])


def accept_tree(target, tokens, parent, u, n):
    """One request: accepted node, path, next token."""
    if n <= 0 or parent[0] != -1 or any(not 0 <= parent[i] < i for i in range(1, n)):
        return -1, [], -1
    V = target.shape[1]
    cur, path, fell, left = 0, [0], [], 1.0
    for i in range(1, n):
        if parent[i] != cur:
            continue
        t = tokens[i]
        p = 0.0 if t in fell or not 0 <= t < V else float(_weights(target[cur, t]))
        if np.float64(u[i]) * left < p:
            cur, fell, left = i, [], 1.0
            path.append(i)
        else:
            left -= p
            fell.append(t)
    p = _weights(target[cur])
    w = p.copy()
    w[[t for t in fell if 0 <= t < V]] = 0
    return cur, path, draw(w if w.any() else p, u[0])


def pool_free(used, table, rows):
    for r in rows:
        if r >= 0 and table[r] >= 0:
            used[table[r]] = 0
            table[r] = -1


def pool_compact(pool, used, table):
    """pool [layers, slots, ...]; all in place; returns the count."""
    count = int(np.count_nonzero(used))
    holes = [s for s in range(count) if not used[s]]
    above = [s for s in range(count, len(used)) if used[s]]
    for d, s in zip(holes, above):
        pool[:, d] = pool[:, s]
        table[table == s] = d
    used[:count], used[count:] = 1, 0
    return count


def pool_fork(pool, used, table, parents, rows):
    """Returns the number of entries that were refused or found no page."""
    before, missed, seen = table.copy(), 0, set()
    was_used = used.copy()
    for p, r in zip(parents, rows):
        if r == -1:
            continue
        if r in seen or before[r] != -1 or (p >= 0 and (before[p] < 0 or not was_used[before[p]])):
            missed += 1
            seen.add(r)
            continue
        seen.add(r)
        free = np.nonzero(used == 0)[0]
        if not len(free):
            missed += 1
            continue
        d = free[0]
        used[d], table[r] = 1, d
        pool[:, d] = pool[:, before[p]] if p >= 0 else 0
    return missed


def lin_decay(rows, a=None, A_log=None, dt_bias=None):
    """Log-decay of every token and value head of linear attention [rows,HV]."""
    if a is None:
        g = np.repeat(-np.exp(np.asarray(A_log, np.float64))[None], rows, 0)
    else:
        g = np.asarray(a, np.float64)[:rows]
        if A_log is not None:
            g = -np.exp(np.asarray(A_log, np.float64)) * np.logaddexp(0, g + (0 if dt_bias is None else np.asarray(dt_bias, np.float64)))
    return np.clip(g, -128, 0)  # a NaN stays one


def lin_unit(x, l2norm):
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6) if l2norm else x


def lin_sequence(S, q, k, v, g, scale, l2norm=True, parents=None):
    """Linear attention over tokens in order (or a tree): S [HV,V,K], q,k [T,H,K],
    v [T,HV,V], log-decays g [T,HV].  Outputs [T,HV,V], states [T,HV,V,K]."""
    S, v = np.asarray(S, np.float64), np.asarray(v, np.float64)
    G = S.shape[0] // q.shape[1]
    q, k = (np.repeat(lin_unit(x, l2norm), G, 1) for x in (q, k))
    states, outs = [], []
    for t in range(len(q)):
        p = t - 1 if parents is None else parents[t]
        S_t = np.exp(g[t])[:, None, None] * (S if p < 0 else states[p]) + v[t][:, :, None] * k[t][:, None, :]
        states.append(S_t)
        outs.append(scale * np.einsum("hvk,hk->hv", S_t, q[t]))
    return np.array(outs), np.array(states)


def logprobs(x, token, top):
    """(log probability, entropy, top tokens, their log probabilities) of one row
    of logits."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, float(np.finfo(np.float32).max)))
    tokens, lps = np.full(top, -1), np.full(top, -np.inf)
    if x.max() == -np.inf:
        return -np.inf, 0.0, tokens, lps
    p = np.exp(x - x.max())
    lp = x - x.max() - np.log(p.sum())
    p /= p.sum()
    order = np.argsort(-x, kind="stable")[:top]
    order = order[x[order] > -np.inf]
    tokens[:len(order)], lps[:len(order)] = order, lp[order]
    return lp[token], -float((p[p > 0] * lp[p > 0]).sum()), tokens, lps


def archived(x, bits):
    """(codes, scales, values read back) of FP32 values x [n, 128]."""
    top, group = (127, 128) if bits == 8 else (7, 32)
    y = np.asarray(x, np.float32).astype(np.float64).reshape(-1, group)
    bad = ~np.isfinite(y).all(1)
    y[bad] = 0
    scale = (np.abs(y).max(1) / top).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(scale[:, None] > 0, np.rint(y / scale.astype(np.float64)[:, None]), 0)
    c = np.clip(c, -top, top)
    scale[bad] = np.nan
    value = c.astype(np.float32) * scale[:, None]
    return c.reshape(x.shape).astype(np.int8), scale.reshape(len(x), -1), value.reshape(x.shape)
