"""The operators together, as examples/speculative_serving.py runs them: the
states that rounds of draft, verify, accept, commit, fork, free and compact
leave behind are those of one prefill over each request's whole text."""
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
