"""The operators together, as examples/speculative_serving.py runs them: the
states that rounds of draft, verify, accept, commit, fork, free and compact
leave behind are those of one prefill over each request's whole text."""
import os
import subprocess
import sys

import pytest
import torch

from examples import speculative_serving as ex
from linear_attention_serving_gated_gb300 import kda
from tests.gpu_util import host_f64, rms

pytestmark = pytest.mark.gpu


def test_rounds_leave_the_states_of_one_prefill():
    s, stood = ex.main()
    stood = torch.cat(stood).cpu()
    assert (stood >= 0).all() and 0 < stood.sum() < 4 * len(stood)  # some drafts stand, some fall
    assert sorted(s.table.tolist()) == [-1, 0, 1, 2] and s.count.item() == 3
    assert s.used.tolist() == [True] * 3 + [False] * 3
    one = ex.Server(s.m, requests=4, slots=4)
    one.start([1, 2, 3], [s.text[r] for r in (1, 2, 3)])
    # Layers see 16-bit rows: a state of later layers differs by what one
    # rounding of its inputs, 2^-8, makes of differences in the layers before.
    # The first layer's rows are those of the prefill, so its states agree as
    # those of decode and prefill do: 2^-12 RMS for the prefill's operands in
    # two halves, and 2^-18 of the largest value a token, 100 tokens.
    got = host_f64(s.pool[:, s.table[1:].long()])
    ref = host_f64(one.pool[:, one.table[1:].long()])
    first = abs(got[0] - ref[0]).max()
    assert first <= 2 ** -12 * rms(ref[0]) + 100 * 2 ** -18 * abs(ref[0]).max()
    assert rms(got[1] - ref[1]) <= 2e-2 * rms(ref[1])
    assert one.err.item() == 0


def test_calls_on_another_stream_own_their_memory():
    """A call on a given stream takes its workspace from that stream's memory:
    what the current stream allocates meanwhile is other memory."""
    m = ex.Model(layers=1)
    d, T = m.d, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k = (torch.randn(T, d.H, 128, generator=g, device="cuda").to(ex.BF16) for _ in range(2))
    v = torch.randn(T, d.HV, 128, generator=g, device="cuda").to(ex.BF16)
    a, b = (torch.randn(T, d.HV, generator=g, device="cuda").to(ex.BF16) for _ in range(2))
    idx = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out = []
    side = torch.cuda.Stream()
    for stream in (None, side):
        pool, o = torch.zeros(1, d.HV, 128, 128, device="cuda"), torch.zeros(T, d.HV, 128, dtype=ex.BF16, device="cuda")
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(2_000_000)  # about a millisecond
        kda.kda_gdn_prefill(d, m.gates[0], q, k, v, a, b, pool, idx, cu, 1, o, stream=stream)
        size = kda.kda_gdn_prefill_workspace_size(d, 1, T)
        torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        out.append((pool, o))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_forms_first_met_under_capture():
    """One small call of a prefill and of an accept, in a process of its own, and
    then other shapes, types and forms of both for the first time under capture."""
    code = """
import torch
from linear_attention_serving_gated_gb300 import kda
torch.manual_seed(0)
def prefill(lengths, H, HV, dt):
    T = sum(lengths)
    d = kda.dims(H, HV=HV, dtype=kda.KDA_DTYPE_F16 if dt is torch.float16 else kda.KDA_DTYPE_BF16)
    x = [torch.randn(T, h, 128, device="cuda").to(dt) for h in (H, H, HV)] + [-torch.rand(T, HV, device="cuda"),
                                                                               torch.randn(T, HV, device="cuda").to(dt)]
    pool = torch.randn(len(lengths), HV, 128, 128, device="cuda") * 0.02
    idx = torch.arange(len(lengths), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + lengths).cumsum(0).int().cuda()
    o = torch.empty(T, HV, 128, dtype=dt, device="cuda")
    ws = torch.empty(kda.kda_gdn_prefill_workspace_size(d, len(lengths), T), dtype=torch.uint8, device="cuda")
    start = pool.clone()
    def run():
        pool.copy_(start)
        kda.kda_gdn_prefill(d, kda.ScalarGate(), *x, pool, idx, cu, len(lengths), o, workspace=ws)
    return run, (pool, o)
def accept(V, dt):
    p = torch.rand(2, 4, V, device="cuda").to(dt)
    tokens = torch.randint(0, V, (2, 4), dtype=torch.int32, device="cuda")
    u = torch.rand(2, 4, device="cuda")
    out = [torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(2)]
    return (lambda: kda.kda_accept_chain(p, None, tokens, u, *out)), out
prefill([3], 1, 1, torch.bfloat16)[0]()
accept(64, torch.float32)[0]()
cases = [prefill(*c) for c in (([70], 8, 16, torch.float16), ([70, 9], 8, 16, torch.bfloat16), ([70] * 9, 8, 16, torch.bfloat16),
                               ([70] * 130, 1, 2, torch.float16))]
cases += [accept(64, torch.float16), accept(512, torch.bfloat16)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for run, _ in cases:
        run()
g.replay()
torch.cuda.synchronize()
for run, out in cases:
    got = [t.clone() for t in out]
    run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, out))
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
