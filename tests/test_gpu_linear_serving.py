"""Linear attention, log probabilities and the archive together, as
examples/speculative_serving.py runs them: prompts, drafts, verification, accept,
commit, fork, a request that waits in the archive, free and compact."""
import numpy as np
import pytest
import torch

from examples import speculative_serving as ex
from linear_attention_serving_gated_gb300 import kda
from tests.gpu_util import host_f64, rms

pytestmark = pytest.mark.gpu


def test_rounds_of_linear_attention(monkeypatch):
    scored, loaded = [], []
    logprobs, load = kda.kda_token_logprobs, kda.kda_pool_load

    def score(logits, tokens, out, **kw):
        logprobs(logits, tokens, out, **kw)
        scored.append([x.clone() for x in (logits, tokens, out, kw["top_tokens"], kw["top_logprobs"])])

    def park(self, rows):
        loaded.append(self.pool[:, self.table[rows].long()].clone())
        stock(self, rows)

    def resume(codes, scales, pool, src, dst, **kw):
        load(codes, scales, pool, src, dst, **kw)
        loaded.append(pool[:, dst.long()].clone())

    stock = ex.Server.park
    monkeypatch.setattr(kda, "kda_token_logprobs", score)
    monkeypatch.setattr(kda, "kda_pool_load", resume)
    monkeypatch.setattr(ex.Server, "park", park)
    s, stood = ex.main(linear=True)
    assert s.err.item() == 0
    stood = torch.cat(stood).cpu()
    assert (stood >= 0).all() and 0 < stood.sum() < 4 * len(stood)
    assert s.count.item() == 2 and sorted(s.table.tolist()) == [-1, 0, 1, 2]  # packed while one waited

    # a state comes back within half a scale, 1/254 of its group's largest value (and an
    # FP32 rounding of the product code * scale)
    before, after = (host_f64(x) for x in loaded)
    half = np.abs(before).max(-1, keepdims=True) / 254
    assert (np.abs(after - before) <= half * (1 + 2.0 ** -20)).all() and rms(after - before) > 0

    # log probabilities of the logits they were asked of: FP32 sums of 512 terms, each
    # exponential within 2^-21: 2^-18 of a log, which is at most 6.3 above the largest, and a
    # difference of numbers below 2^6 rounded to 2^-18
    for logits, tokens, out, tops, top_scores in scored:
        ref = torch.log_softmax(logits.double(), -1)
        ok = tokens >= 0
        want = ref.gather(1, tokens.clamp(min=0).long()[:, None])[:, 0]
        assert (logits.abs() < 64).all() and ((out - want).abs() <= 2.0 ** -16)[ok].all() and (out[~ok] == 0).all()
        best = logits.topk(3, -1)
        assert torch.equal(logits.gather(1, tops.clamp(min=0).long())[ok], best.values[ok])
        assert ((top_scores - ref.gather(1, best.indices)).abs() <= 2.0 ** -16)[ok].all()
    prompts = {0: 1, 1: 70, 2: 33}
    for r in (1, 2):
        assert len(s.scores[r]) == len(s.text[r]) - prompts[r] + 1

    # requests that never waited: the first layer's states are those of one prefill
    # over the whole text, as for the other rule
    one = ex.Server(s.m, requests=4, slots=4)
    one.start([1, 3], [s.text[r] for r in (1, 3)])
    got, ref = (host_f64(x.pool[:, x.table[[1, 3]].long()]) for x in (s, one))
    assert abs(got[0] - ref[0]).max() <= 2 ** -12 * rms(ref[0]) + 100 * 2 ** -18 * abs(ref[0]).max()
    assert rms(got[1] - ref[1]) <= 2e-2 * rms(ref[1])
    assert one.err.item() == 0


def calls():
    """Entry point -> (its call, what it writes, what that holds before)."""
    torch.manual_seed(0)
    T, H = 200, 2
    rows = lambda n, h, dt=torch.bfloat16: torch.randn(n, h, 128, device="cuda").to(dt)  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    gate = kda.ScalarGate()
    fixed = kda.ScalarGate(A_log=torch.zeros(H, device="cuda"))
    pool, idx, cu = torch.randn(4, H, 128, 128, device="cuda") * 0.02, i32(2, 0), i32(0, 70, T)
    a = -torch.rand(T, H, device="cuda")
    out = {}
    for name, dt, code in (("bf16", torch.bfloat16, kda.KDA_DTYPE_BF16), ("f16", torch.float16, kda.KDA_DTYPE_F16)):
        d, x, o = kda.dims(H, dtype=code), [rows(T, H, dt) for _ in "qkv"], torch.zeros(T, H, 128, dtype=dt, device="cuda")
        out["kda_lin_prefill " + name] = (lambda d=d, x=x, o=o: kda.kda_lin_prefill(d, gate, *x, a, pool, idx, cu, 2, o), (o, pool))
    long = [rows(4096, 1) for _ in "qkv"]
    lo, lcu = torch.zeros(4096, 1, 128, dtype=torch.bfloat16, device="cuda"), i32(0, 4096)
    lpool, one, lidx = torch.randn(1, 1, 128, 128, device="cuda"), kda.dims(1), i32(0)
    slow = kda.ScalarGate(A_log=torch.zeros(1, device="cuda") - 4)
    out["kda_lin_prefill in segments"] = (lambda: kda.kda_lin_prefill(
        one, slow, *long, None, lpool, lidx, lcu, 1, lo), (lo, lpool))
    d = kda.dims(H)
    packed = rows(6, 3 * H).flatten(1)
    o2, o6 = (torch.zeros(n, H, 128, dtype=torch.bfloat16, device="cuda") for n in (2, 6))
    snaps = torch.zeros(2, 3, H, 128, 128, device="cuda")
    out["kda_lin_decode_packed"] = (lambda: kda.kda_lin_decode_packed(d, gate, packed[:2], a[:2], pool, idx, o2), (o2, pool))
    out["kda_lin_verify_chain"] = (lambda: kda.kda_lin_verify_chain(d, fixed, packed, None, 2, 3, pool, idx, o6, snaps), (o6, snaps))
    parents = i32(-1, 0, 0, -1, 0, 1)
    out["kda_lin_verify_tree"] = (lambda: kda.kda_lin_verify_tree(d, gate, packed, a[:6], 2, 3, parents, pool, idx, o6, snaps),
                                  (o6, snaps))
    logits = torch.randn(3, 5000, device="cuda") * 3
    lp, ent, tt, tl = (torch.zeros(*s, dtype=t, device="cuda") for s, t in (((3,), torch.float32), ((3,), torch.float32),
                                                                           ((3, 4), torch.int32), ((3, 4), torch.float32)))
    tok = i32(7, -1, 4999)
    out["kda_token_logprobs"] = (lambda: kda.kda_token_logprobs(logits, tok, lp, ent, tt, tl), (lp, ent, tt, tl))
    pages = torch.randn(2, 8, 4096, device="cuda")
    src, dst = i32(6, 1), i32(0, 2)
    for bits, t, n in ((8, torch.int8, 4096), (4, torch.uint8, 2048)):
        codes = torch.zeros(3, 2, n, dtype=t, device="cuda")
        scales = torch.zeros(3, 2, 32 if bits == 8 else 128, device="cuda")
        out[f"kda_pool_store {bits}"] = (lambda c=codes, s=scales: kda.kda_pool_store(pages, c, s, src, dst), (codes, scales))
        full, fs = torch.randint(0, 100, codes.shape, device="cuda").to(t), torch.rand_like(scales)
        out[f"kda_pool_load {bits}"] = (lambda c=full, s=fs: kda.kda_pool_load(c, s, pages, dst, src), (pages,))
    return out


NAMES = ["kda_lin_prefill bf16", "kda_lin_prefill f16", "kda_lin_prefill in segments", "kda_lin_decode_packed",
         "kda_lin_verify_chain", "kda_lin_verify_tree", "kda_token_logprobs", "kda_pool_store 8", "kda_pool_store 4",
         "kda_pool_load 8", "kda_pool_load 4"]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_stage_events(name, captured):
    """Every entry point with stage events set, eagerly and captured, gives what it
    gives without, and records them in order."""
    call, outs = calls()[name]
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    call, outs = calls()[name]
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for e in ev:
        e.record()
    torch.cuda.synchronize()
    try:
        kda.kda_set_stage_events(ev)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            graph.replay()
        else:
            call()
    finally:
        kda.kda_set_stage_events(None)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want))
    assert ev[0].elapsed_time(ev[2]) > 0 and ev[0].elapsed_time(ev[1]) >= 0 and ev[1].elapsed_time(ev[2]) >= 0


def test_two_streams_at_once():
    """Every call twice at the same time, on streams of their own with data of their own,
    again and again, gives what it gives alone."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    for name in NAMES:
        want = []
        call, outs = calls()[name]
        for _ in range(3):  # some calls go on from what the last left
            call()
        torch.cuda.synchronize()
        want = [x.clone() for x in outs]
        sets = [calls()[name] for _ in sides]
        torch.cuda.synchronize()
        for _ in range(3):
            for side, (call, _) in zip(sides, sets):
                with torch.cuda.stream(side):
                    call()
        torch.cuda.synchronize()
        for _, outs in sets:
            assert all(torch.equal(x, y) for x, y in zip(outs, want)), name


def test_forms_first_met_under_capture():
    """A small call of each, in a process of its own, and then other types, sizes and
    forms for the first time under capture."""
    import os
    import subprocess
    import sys

    code = """
import torch
from linear_attention_serving_gated_gb300 import kda
from tests import test_gpu_linear_serving as t
def logits(dt, rows, vocab, top):
    x = torch.randn(rows, vocab, device="cuda").to(dt)
    out = [torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, top, dtype=torch.int32, device="cuda"),
           torch.empty(rows, top, device="cuda")]
    tok = torch.zeros(rows, dtype=torch.int32, device="cuda")
    return (lambda: kda.kda_token_logprobs(x, tok, *(out if top else out[:2]))), out if top else out[:2]
first = t.calls()
for name in ("kda_lin_prefill bf16", "kda_lin_decode_packed", "kda_token_logprobs", "kda_pool_store 8"):
    first[name][0]()
cases = [t.calls()[name] for name in t.NAMES]
cases += [logits(dt, r, v, top) for dt in (torch.float32, torch.bfloat16, torch.float16) for r, v, top in
          ((1, 70000, 32), (400, 3000, 0), (5, 33, 1), (2, 300000, 8))]
torch.cuda.synchronize()
starts = [[x.clone() for x in outs] for _, outs in cases]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for call, _ in cases:
        call()
g.replay()
torch.cuda.synchronize()
for (call, outs), start in zip(cases, starts):
    got = [x.clone() for x in outs]
    for x, y in zip(outs, start):
        x.copy_(y)
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, outs))
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
