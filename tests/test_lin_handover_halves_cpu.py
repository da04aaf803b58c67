"""The hand-overs of csrc/lin_prefill.cu's second launch, where the state's operand and P have
one place each, handed over together, that their products must have read before the next
chunk's go there.  The model's machinery, and its other programs, are those of
test_lin_handover_cpu.py; the order of waits and arrivals is compared with the kernel's."""
import os
import re

import pytest

from linear_attention_serving_gated_gb300 import build
from tests import test_lin_handover_cpu as model

BUFS, STAGES = model.BUFS, model.STAGES


def worker(t, w, early=False):
    """early: the operand is stored before the last one's product is waited for."""
    if t.local:
        yield from model_worker(t, w)
        return
    n = t.nch

    def keys(c):
        yield ("in", c % BUFS), c // BUFS
        t.use_factors(c)
        t.use(("K", c % STAGES), c)
        if w == 0:
            t.put(("V", c % STAGES), c)
        t.put(("wk", 0, w), c)

    def outputs(c):
        t.use(("O1", c & 1), c)
        t.use(("O2", c & 1), c)
        t.use_factors(c)
        yield
        t.bar["free", c % BUFS].arrive()

    yield from keys(0)
    yield
    t.bar["wk", 0].arrive()
    if t.pool:
        yield ("state", 0), 0
        for place in t.state:
            t.use(place, "state")
            yield
        t.bar["met", 0].arrive()
        yield ("met", 0), 0
        if w == 0:
            t.bar["read", 0].arrive()
    for c in range(n):
        if c > 0:
            t.use(("dS", 0), c - 1)
            yield
            t.use(("dS", 0), c - 1)
        t.bar["u", 0].arrive()
        yield
        t.use_factors(c)
        yield
        if early:
            t.put(("S", 0, w), c)
            yield
        if c > 0:
            yield ("o", 0), c - 1
        t.put(("S", 0, w), c)
        yield
        yield ("qk", 0), c
        t.use(("QK", c & 1), c)
        t.use_factors(c)
        yield
        t.put(("P", w), c)
        yield
        t.bar["p", 0].arrive()
        yield
        if c > 0:
            yield from outputs(c - 1)
        yield ("ds", c & 1), c >> 1
        if c + 1 < n:
            yield from keys(c + 1)
            yield
            t.bar["wk", (c + 1) & 1].arrive()
        yield
    yield ("o", 0), n - 1
    yield from outputs(n - 1)
    t.use(("dS", 0), n - 1)


def products(t):
    if t.local:
        yield from model_products(t)
        return
    W = range(t.workers)
    for c in range(t.nch):
        st = c % STAGES
        yield ("in", c % BUFS), c // BUFS
        yield ("wk", c & 1), c >> 1
        t.product([("Q", st), ("K", st)], [("QK", c & 1)], c)
        t.commit(("qk", 0))
        yield ("u", 0), c
        t.product([("V", st)] + [("wk", 0, x) for x in W], [("dS", 0)], c)
        t.commit(("ds", c & 1))
        yield ("p", 0), c
        t.product([("Q", st)] + [("S", 0, x) for x in W], [("O1", c & 1)], c)
        t.product([("V", st)] + [("P", x) for x in W], [("O2", c & 1)], c)
        t.commit(("empty", st))
        t.commit(("o", 0))
        yield


model_worker, model_products = model.worker, model.products


@pytest.mark.parametrize("local", [False, True])
@pytest.mark.parametrize("nch", [1, 2, 3, 4, 5, 9, 20])
def test_every_order_ends_and_overwrites_nothing(nch, local, monkeypatch):
    monkeypatch.setattr(model, "worker", worker)
    monkeypatch.setattr(model, "products", products)
    for seed in range(150):
        model.run(nch, local, seed)


def test_the_model_sees_an_operand_overwritten(monkeypatch):
    monkeypatch.setattr(model, "worker", lambda t, w: worker(t, w, early=True))
    monkeypatch.setattr(model, "products", products)
    with pytest.raises(AssertionError, match="overwritten|holds"):
        for seed in range(150):
            model.run(9, False, seed)


def test_the_kernel_waits_and_arrives_in_the_models_order():
    with open(os.path.join(build.CSRC, "lin_prefill.cu")) as f:
        source = f.read()

    def steps(start, end):
        part = source[source.index(start):]
        part = re.sub(r"//[^\n]*", "", part[:part.index(end)])
        return [" ".join(x) for x in re.findall(r"\b(warp_wait|await|done|mma_commit|keys|update|operand|weights|outputs)\((?:&bars\.(\w+))?", part)]

    assert steps("auto weights = ", "// ---") == ["await qk_full", "operand ", "operand ", "done p_full"]
    assert steps("const uint64_t wk_op = tc::sw128_desc_mn(tc::smem_u32(smem + kWk)", "} else if (warp < kNormWarp)") == [
        "warp_wait in_full", "warp_wait wk_full", "mma_commit qk_full", "warp_wait u_full", "mma_commit ds_full", "warp_wait p_full",
        "mma_commit empty", "mma_commit o_full"]
    loop = source[source.index("if (LOCAL) {\n      // K' and dS are there twice"):]
    source = loop[loop.index("} else {"):]
    assert steps("for (int c = 0", "if (LOCAL) await") == [
        "update ", "done u_full", "await o_full", "operand ", "weights ", "outputs ", "await ds_full", "keys ", "done wk_full",
        "await o_full", "outputs "]
