"""Speculative serving of a small random-weight model whose layers are the gated
delta rule with one decay per value head: prompts are prefilled into pages of a
state pool, every round verifies drafted tokens in one pass, keeps those that
stand and commits their states, a request forks into two, another ends and
leaves its pages, and the pool is packed again.  Every token of the text has its
log probability under the model.  `linear` takes plain linear attention with one
decay per head for the rule, and one request's state waits in 8 bits meanwhile.

    python examples/speculative_serving.py [linear]

The draft is the target distribution, flattened: good enough that tokens stand
and bad enough that tokens fall.  All indices stay on the device; the host
reads a round's result only to keep the text.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_attention_serving_gated_gb300 import kda  # noqa: E402

K = V = 128
BF16 = torch.bfloat16


class Model:
    """Embedding, `layers` of (projections, delta rule, output projection) and
    a head; `linear`: linear attention for the delta rule."""

    def __init__(self, layers=2, H=2, HV=4, vocab=512, width=256, device="cuda", seed=0, linear=False):
        g = torch.Generator(device=device).manual_seed(seed)
        draw = lambda *s: torch.randn(*s, generator=g, device=device) * s[-1] ** -0.5  # noqa: E731
        self.layers, self.vocab, self.d, self.linear = layers, vocab, kda.dims(H, HV=HV), linear
        self.qkv = 2 * H * K + HV * V
        self.embed = draw(vocab, width) * width ** 0.5
        self.head = draw(vocab, width) * 4
        self.w_in = [draw(self.qkv + 2 * HV, width) for _ in range(layers)]
        self.w_out = [draw(width, HV * V) for _ in range(layers)]
        self.gates = [kda.ScalarGate(A_log=torch.empty(HV, device=device).uniform_(0, 2, generator=g),
                                     dt_bias=torch.empty(HV, device=device).uniform_(-6, -2, generator=g))
                      for _ in range(layers)]

    @staticmethod
    def _norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def call(self, name, l, rows, gates, *rest, **kw):
        """Layer l's kda_gdn_<name> or kda_lin_<name>."""
        gates = gates[:1] if self.linear else gates  # (a, b): linear attention has no b
        getattr(kda, ("kda_lin_" if self.linear else "kda_gdn_") + name)(self.d, self.gates[l], *rows, *gates, *rest, **kw)

    def run(self, tokens, rule):
        """Logits behind `tokens`; rule(layer, packed rows, (a, b), o) is one of the
        calls on the states."""
        x = self.embed[tokens]
        for l in range(self.layers):
            y = self._norm(x) @ self.w_in[l].T
            qkv, a, b = y.to(BF16).split((self.qkv, self.d.HV, self.d.HV), dim=-1)
            o = torch.empty(len(tokens), self.d.HV, V, dtype=BF16, device=x.device)
            rule(l, qkv.contiguous(), (a.contiguous(), b.contiguous()), o)
            x = x + o.flatten(1).float() @ self.w_out[l].T
        return self._norm(x) @ self.head.T


class Server:
    def __init__(self, model, requests, slots, device="cuda"):
        self.m, self.err = model, torch.zeros(1, dtype=torch.int32, device=device)
        d = model.d
        self.pool = torch.zeros(model.layers, slots, d.HV, V, K, device=device)
        self.used = torch.zeros(slots, dtype=torch.bool, device=device)
        self.table = torch.full((requests,), -1, dtype=torch.int32, device=device)  # row of a request -> slot
        self.count = torch.zeros(1, dtype=torch.int32, device=device)
        self.next = torch.zeros(requests, dtype=torch.int32, device=device)  # sampled, not yet in the state
        self.text = [[] for _ in range(requests)]
        self.scores = [[] for _ in range(requests)]  # log probabilities of the tokens behind a prompt, and of `next`
        page = (model.layers, d.HV, V, K)
        self.codes = torch.zeros(requests, *page, dtype=torch.int8, device=device)  # pages that wait, by request
        self.scales = torch.zeros(requests, *page[:-1], 1, device=device)
        self.g = torch.Generator(device=device).manual_seed(1)

    def _rows(self, rows):
        return torch.tensor(rows, dtype=torch.int32, device=self.pool.device)

    def start(self, rows, prompts):
        """Empty pages for new requests, and their prompts' states."""
        m, d, dev = self.m, self.m.d, self.pool.device
        kda.kda_pool_fork(self.pool, self.used, self.table, self._rows([-1] * len(rows)), self._rows(rows),
                          err_flag=self.err)
        idx = self.table[self._rows(rows)]
        ends = torch.tensor([0] + [len(p) for p in prompts]).cumsum(0)
        cu = ends.to(torch.int32).to(dev)

        def rule(l, qkv, gates, o):
            q, k, v = (x.contiguous() for x in qkv.split((d.H * K, d.H * K, d.HV * V), dim=-1))
            m.call("prefill", l, (q, k, v), gates, self.pool[l], idx, cu, len(rows), o, err_flag=self.err)

        last = m.run(torch.tensor([t for x in prompts for t in x], device=dev), rule)[ends[1:].to(dev) - 1]
        after = torch.softmax(last, dim=-1).argmax(-1).int()
        self.next[self._rows(rows)] = after
        for r, x, score in zip(rows, prompts, self.score(last, after)[0].tolist()):
            self.text[r], self.scores[r] = list(x), [score]

    def score(self, logits, tokens, top=3):
        """Log probabilities of tokens [rows] and the `top` alternatives and theirs."""
        rows, dev = len(tokens), logits.device
        out = torch.empty(rows, device=dev)
        top_tokens, top_scores = torch.empty(rows, top, dtype=torch.int32, device=dev), torch.empty(rows, top, device=dev)
        kda.kda_token_logprobs(logits, tokens, out, top_tokens=top_tokens, top_logprobs=top_scores, err_flag=self.err)
        return out, top_tokens, top_scores

    def draft(self, idx, tokens, T):
        """T - 1 tokens behind tokens [B] and their distributions, one decode
        each on a copy of the states."""
        m, scratch = self.m, self.pool.clone()
        out, probs = [tokens], []
        for _ in range(T - 1):
            p = torch.softmax(m.run(out[-1], lambda l, qkv, gates, o: m.call(
                "decode_packed", l, (qkv,), gates, scratch[l], idx, o, err_flag=self.err)), dim=-1)
            p = p.sqrt()
            probs.append(p / p.sum(-1, keepdim=True))
            out.append(torch.multinomial(probs[-1], 1, generator=self.g)[:, 0].int())
        return torch.stack(out, 1), torch.stack(probs, 1)

    def round(self, rows, T=5):
        """Draft, verify, keep what stands, commit."""
        m, d, dev, B = self.m, self.m.d, self.pool.device, len(rows)
        r = self._rows(rows)
        idx = self.table[r]
        tokens, q = self.draft(idx, self.next[r], T)
        snaps = torch.empty(m.layers, B, T, d.HV, V, K, device=dev)
        logits = m.run(tokens.flatten(), lambda l, qkv, gates, o: m.call(
            "verify_chain", l, (qkv,), gates, B, T, self.pool[l], idx, o, snaps[l], err_flag=self.err))
        p = torch.softmax(logits, dim=-1)
        accepted, after = torch.empty_like(r), torch.empty_like(r)
        kda.kda_accept_chain(p.view(B, T, -1), q, tokens, torch.rand(B, T, generator=self.g, device=dev), accepted,
                             after, err_flag=self.err)
        for l in range(m.layers):
            kda.kda_commit(d, snaps[l], B, T, accepted, self.pool[l], idx, err_flag=self.err)
        self.next[r] = after
        at = torch.arange(T, device=dev)  # behind token t stands the next draft, or what was drawn, or nothing
        behind = torch.cat([tokens[:, 1:], tokens[:, :1]], 1)
        behind = torch.where(at < accepted[:, None], behind, torch.where(at == accepted[:, None], after[:, None], -1))
        scores = self.score(logits, behind.flatten())[0].view(B, T)
        for row, n, line, score in zip(rows, accepted.tolist(), tokens.tolist(), scores.tolist()):
            self.text[row] += line[:n + 1]
            self.scores[row] += score[:n + 1]
        return accepted

    def fork(self, row, child):
        """Request `child` goes on from where `row` is."""
        kda.kda_pool_fork(self.pool, self.used, self.table, self._rows([row]), self._rows([child]),
                          err_flag=self.err)
        self.next[child] = self.next[row]
        self.text[child], self.scores[child] = list(self.text[row]), list(self.scores[row])

    def park(self, rows):
        """Requests that wait leave the pool; their states stay, in 8 bits."""
        kda.kda_pool_store(self.pool, self.codes, self.scales, self.table[self._rows(rows)], self._rows(rows),
                           err_flag=self.err)
        self.finish(rows)

    def resume(self, rows):
        """Their states come back, into pages of their own."""
        r = self._rows(rows)
        kda.kda_pool_fork(self.pool, self.used, self.table, self._rows([-1] * len(rows)), r, err_flag=self.err)
        kda.kda_pool_load(self.codes, self.scales, self.pool, r, self.table[r], err_flag=self.err)

    def finish(self, rows):
        """The pages of ended requests become free, and the used ones move
        together."""
        kda.kda_pool_free(self.used, self.table, self._rows(rows), err_flag=self.err)
        kda.kda_pool_compact(self.pool, self.used, self.table, self.count, err_flag=self.err)


def main(device="cuda", linear=False):
    g = torch.Generator().manual_seed(2)
    model = Model(device=device, linear=linear)
    s = Server(model, requests=4, slots=6, device=device)
    s.start([0, 1, 2], [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in (1, 70, 33)])
    stood = [s.round([0, 1, 2]) for _ in range(3)]
    s.fork(1, 3)
    stood.append(s.round([0, 1, 2, 3]))
    s.finish([0])
    if linear:
        s.park([2])
        stood.append(s.round([1, 3]))
        s.resume([2])
    stood += [s.round([1, 2, 3]) for _ in range(2)]
    if s.err.item():
        raise RuntimeError(f"error bits {s.err.item()}")
    print("drafts that stood, of 4 per round:", [x.tolist() for x in stood])
    for r in (1, 2, 3):
        print(f"request {r}: slot {s.table[r].item()}, {len(s.text[r])} tokens, the last {s.text[r][-8:]}, "
              f"log probability a token {sum(s.scores[r]) / len(s.scores[r]):.2f}")
    return s, stood


if __name__ == "__main__":
    main(linear="linear" in sys.argv[1:])
