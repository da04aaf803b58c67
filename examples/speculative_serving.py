"""Speculative serving of a small random-weight model whose layers are the gated
delta rule with one decay per value head: prompts are prefilled into pages of a
state pool, every round verifies drafted tokens in one pass, keeps those that
stand and commits their states, a request forks into two, another ends and
leaves its pages, and the pool is packed again.

    python examples/speculative_serving.py

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
    a head."""

    def __init__(self, layers=2, H=2, HV=4, vocab=512, width=256, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        draw = lambda *s: torch.randn(*s, generator=g, device=device) * s[-1] ** -0.5  # noqa: E731
        self.layers, self.vocab, self.d = layers, vocab, kda.dims(H, HV=HV)
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

    def run(self, tokens, rule):
        """Probabilities behind `tokens`; rule(layer, packed rows, a, b, o) is
        one of the calls on the states."""
        x = self.embed[tokens]
        for l in range(self.layers):
            y = self._norm(x) @ self.w_in[l].T
            qkv, a, b = y.to(BF16).split((self.qkv, self.d.HV, self.d.HV), dim=-1)
            o = torch.empty(len(tokens), self.d.HV, V, dtype=BF16, device=x.device)
            rule(l, qkv.contiguous(), a.contiguous(), b.contiguous(), o)
            x = x + o.flatten(1).float() @ self.w_out[l].T
        return torch.softmax(self._norm(x) @ self.head.T, dim=-1)


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

        def rule(l, qkv, a, b, o):
            q, k, v = (x.contiguous() for x in qkv.split((d.H * K, d.H * K, d.HV * V), dim=-1))
            kda.kda_gdn_prefill(d, m.gates[l], q, k, v, a, b, self.pool[l], idx, cu, len(rows), o, err_flag=self.err)

        p = m.run(torch.tensor([t for x in prompts for t in x], device=dev), rule)
        self.next[self._rows(rows)] = p[ends[1:].to(dev) - 1].argmax(-1).int()
        for r, x in zip(rows, prompts):
            self.text[r] = list(x)

    def draft(self, idx, tokens, T):
        """T - 1 tokens behind tokens [B] and their distributions, one decode
        each on a copy of the states."""
        m, scratch = self.m, self.pool.clone()
        out, probs = [tokens], []
        for _ in range(T - 1):
            p = m.run(out[-1], lambda l, qkv, a, b, o: kda.kda_gdn_decode_packed(
                m.d, m.gates[l], qkv, a, b, scratch[l], idx, o, err_flag=self.err))
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
        p = m.run(tokens.flatten(), lambda l, qkv, a, b, o: kda.kda_gdn_verify_chain(
            d, m.gates[l], qkv, a, b, B, T, self.pool[l], idx, o, snaps[l], err_flag=self.err))
        accepted, after = torch.empty_like(r), torch.empty_like(r)
        kda.kda_accept_chain(p.view(B, T, -1), q, tokens, torch.rand(B, T, generator=self.g, device=dev), accepted,
                             after, err_flag=self.err)
        for l in range(m.layers):
            kda.kda_commit(d, snaps[l], B, T, accepted, self.pool[l], idx, err_flag=self.err)
        self.next[r] = after
        for row, n, line in zip(rows, accepted.tolist(), tokens.tolist()):
            self.text[row] += line[:n + 1]
        return accepted

    def fork(self, row, child):
        """Request `child` goes on from where `row` is."""
        kda.kda_pool_fork(self.pool, self.used, self.table, self._rows([row]), self._rows([child]),
                          err_flag=self.err)
        self.next[child] = self.next[row]
        self.text[child] = list(self.text[row])

    def finish(self, rows):
        """The pages of ended requests become free, and the used ones move
        together."""
        kda.kda_pool_free(self.used, self.table, self._rows(rows), err_flag=self.err)
        kda.kda_pool_compact(self.pool, self.used, self.table, self.count, err_flag=self.err)


def main(device="cuda"):
    g = torch.Generator().manual_seed(2)
    model = Model(device=device)
    s = Server(model, requests=4, slots=6, device=device)
    s.start([0, 1, 2], [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in (1, 70, 33)])
    stood = [s.round([0, 1, 2]) for _ in range(3)]
    s.fork(1, 3)
    stood.append(s.round([0, 1, 2, 3]))
    s.finish([0])
    stood += [s.round([1, 2, 3]) for _ in range(2)]
    if s.err.item():
        raise RuntimeError(f"error bits {s.err.item()}")
    print("drafts that stood, of 4 per round:", [x.tolist() for x in stood])
    for r in (1, 2, 3):
        print(f"request {r}: slot {s.table[r].item()}, {len(s.text[r])} tokens, the last {s.text[r][-8:]}")
    return s, stood


if __name__ == "__main__":
    main()
