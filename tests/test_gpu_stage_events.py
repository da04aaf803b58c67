"""Stage events (kda_set_stage_events): every entry point runs with them set,
launched eagerly and captured, gives what it gives without, and records them in
order."""
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda

pytestmark = pytest.mark.gpu
K = 128


def rows(T, heads, dt=torch.bfloat16):
    return torch.randn(T, heads, K, device="cuda").to(dt)


def calls():
    """Entry point -> (its call, what it writes)."""
    torch.manual_seed(0)
    T, H = 200, 2
    d, f16 = kda.dims(H), kda.dims(H, dtype=kda.KDA_DTYPE_F16)
    gate = kda.ScalarGate()
    pool = torch.randn(4, H, K, K, device="cuda") * 0.02
    idx = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 70, T], dtype=torch.int32, device="cuda")
    g, b = -torch.rand(T, H, device="cuda"), torch.randn(T, H, device="cuda").bfloat16()
    q, k, v = rows(T, H), rows(T, H), rows(T, H)
    o = torch.zeros(T, H, K, dtype=torch.bfloat16, device="cuda")
    packed = rows(2, 3 * H).flatten(1)
    od = torch.zeros(2, H, K, dtype=torch.bfloat16, device="cuda")
    kg = kda.Gate(A_log=torch.zeros(H, device="cuda"), dt_bias=torch.zeros(H * K, device="cuda"))
    kg_in = torch.randn(T, H, K, device="cuda").bfloat16()
    hq, hk, hv, hb = (x.half() for x in (q, k, v, b))
    ho = o.half()
    pages = torch.randn(2, 8, 4096, device="cuda")
    used = torch.tensor([0, 1, 0, 1, 1, 0, 1, 0], dtype=torch.uint8, device="cuda")
    table = torch.tensor([6, 3, 1, 4, -1], dtype=torch.int32, device="cuda")
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    par, row, kids = i32(0), i32(4), i32(0)
    p, tok, u = torch.softmax(torch.randn(2, 3, 1000, device="cuda"), -1), i32(1, 2, 3, 4, 5, 6).view(2, 3), torch.rand(
        2, 3, device="cuda")
    acc, nxt = i32(0, 0), i32(0, 0)
    return {
        "kda_prefill": (lambda: kda.kda_prefill(d, kg, q, k, v, kg_in, b, pool, idx, cu, 2, o), (o, pool)),
        "kda_gdn_prefill": (lambda: kda.kda_gdn_prefill(d, gate, q, k, v, g, b, pool, idx, cu, 2, o), (o, pool)),
        "kda_gdn_prefill f16": (lambda: kda.kda_gdn_prefill(f16, gate, hq, hk, hv, g, hb, pool, idx, cu, 2, ho), (ho, pool)),
        "kda_gdn_decode_packed": (lambda: kda.kda_gdn_decode_packed(d, gate, packed, g[:2], b[:2], pool, idx, od), (od, pool)),
        "kda_accept_chain": (lambda: kda.kda_accept_chain(p, None, tok, u, acc, nxt), (acc, nxt)),
        "kda_pool_compact": (lambda: kda.kda_pool_compact(pages, used, table, count), (pages, used, table, count)),
        "kda_pool_fork": (lambda: kda.kda_pool_fork(pages, used, table, par, row, children=kids), (pages, used, table, kids)),
    }


NAMES = ["kda_prefill", "kda_gdn_prefill", "kda_gdn_prefill f16", "kda_gdn_decode_packed", "kda_accept_chain", "kda_pool_compact",
         "kda_pool_fork"]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_stage_events(name, captured):
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
