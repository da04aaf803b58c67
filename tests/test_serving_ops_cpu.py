"""Refusals of the serving operators that need no GPU: host status codes of the
C ABI (every call returns before it touches the device) and the binding's shape
and type rules; and the oracle's own invariants."""
import ctypes

import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import build, kda
from oracle import serving_oracle as so

D = ctypes.c_void_p(0x10000)  # never dereferenced
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kda.load()


def sgate(A_log=D):
    return kda.kda_scalar_gate(A_log, None, 1, 1, 128 ** -0.5)


def test_gdn_host_errors(lib):
    row = 3 * 16 * 128

    def pre(d=kda.dims(16), g=sgate(), q=D, a=D, pool=D, idx=D, gb=64, T=64, n=1, inter=None, chunks=0,
            ws=D, ws_bytes=1 << 40):
        return lib.kda_gdn_prefill(d, g, q, D, D, a, D, gb, pool, 4, idx, None, n, T, D, inter, chunks, ws, ws_bytes,
                                   None, None)

    assert pre(pool=None) == pre(idx=None) == pre(q=None) == kda.KDA_ERR_NULL_ARG
    assert pre(gb=63) == pre(T=65, gb=65, n=2) == pre(T=2 ** 31, gb=2 ** 31) == kda.KDA_ERR_SHAPE
    assert pre(inter=D, chunks=-1) == pre(n=0) == kda.KDA_ERR_SHAPE
    assert pre(d=kda.dims(4, K=64, V=64)) == pre(d=kda.dims(4, HV=6)) == pre(d=kda.dims(4, dtype=2)) == kda.KDA_ERR_UNSUPPORTED
    assert pre(q=ODD) == pre(pool=ODD) == kda.KDA_ERR_ALIGNMENT
    assert pre(g=sgate(None), a=ODD) == pre(a=ctypes.c_void_p(0x10001)) == kda.KDA_ERR_ALIGNMENT
    assert pre(T=0, gb=0) == kda.KDA_OK  # nothing to do
    f16 = kda.dims(16, dtype=kda.KDA_DTYPE_F16)
    assert kda.kda_gdn_prefill_workspace_size(kda.dims(16), 3, 100) == 4 * 16 * 33792
    assert kda.kda_gdn_prefill_workspace_size(f16, 3, 100) == 4 * 16 * 33792 + 4 * 100 * 16 * 256
    assert kda.kda_gdn_prefill_workspace_size(kda.dims(16), 1, 2 ** 31) == 2 ** 64 - 1
    assert pre(ws=None) == pre(ws_bytes=2 * 16 * 33792 - 1) == kda.KDA_ERR_WORKSPACE
    assert pre(d=f16, ws_bytes=2 * 16 * 33792) == kda.KDA_ERR_WORKSPACE
    assert pre(ws=ODD) == kda.KDA_ERR_ALIGNMENT

    def dec(d=kda.dims(16), stride=row, pool=D, qkv=D, B=2):
        return lib.kda_gdn_decode_packed(d, sgate(), qkv, stride, D, D, B, pool, 240, D, D, None, None)

    assert dec(pool=None) == dec(qkv=None) == kda.KDA_ERR_NULL_ARG
    assert dec(stride=row - 8) == dec(B=-1) == kda.KDA_ERR_SHAPE
    assert dec(stride=row + 4) == dec(qkv=ODD) == kda.KDA_ERR_ALIGNMENT
    assert dec(d=kda.dims(16, HV=24)) == kda.KDA_ERR_UNSUPPORTED
    assert dec(B=0) == kda.KDA_OK
    d = kda.dims(16)
    assert lib.kda_gdn_verify_chain(d, sgate(), D, row, D, D, 2, 0, D, 9, D, D, D, None, None) == kda.KDA_ERR_SHAPE
    assert lib.kda_gdn_verify_chain(d, sgate(), D, row, D, D, 2, 6, D, 9, D, D, None, None, None) == kda.KDA_ERR_NULL_ARG
    assert lib.kda_gdn_verify_tree(d, sgate(), D, row, D, D, 2, 6, None, D, 9, D, D, D, None, None) == kda.KDA_ERR_NULL_ARG
    assert lib.kda_gdn_verify_chain(d, sgate(), D, row, D, D, 2, 6, D, 9, D, D, ODD, None, None) == kda.KDA_ERR_ALIGNMENT


def test_accept_host_errors(lib):
    def chain(dt=2, target=D, stride=100, draft=D, dstride=100, tokens=D, B=2, T=3, V=100, out=D):
        return lib.kda_accept_chain(dt, target, stride, draft, dstride, tokens, D, None, B, T, V, out, D, None, None)

    assert chain(dt=3) == chain(T=1025) == kda.KDA_ERR_UNSUPPORTED
    assert chain(V=(1 << 28) + 1, stride=1 << 30, dstride=1 << 30) == kda.KDA_ERR_UNSUPPORTED
    assert chain(target=None) == chain(tokens=None) == chain(out=None) == kda.KDA_ERR_NULL_ARG
    assert chain(stride=99) == chain(dstride=99) == chain(T=0) == chain(V=0) == chain(B=-1) == kda.KDA_ERR_SHAPE
    assert chain(target=ODD) == chain(draft=ODD) == kda.KDA_ERR_ALIGNMENT
    assert chain(B=0) == kda.KDA_OK
    assert lib.kda_accept_tree(2, D, 100, D, None, D, None, 2, 3, 100, D, D, D, None, None) == kda.KDA_ERR_NULL_ARG
    assert lib.kda_accept_tree(2, D, 100, D, D, D, None, 2, 3, 100, D, None, D, None, None) == kda.KDA_ERR_NULL_ARG


def test_pool_host_errors(lib):
    def pages(base=0x10000, page=1024, stride=8192, layers=2, slots=8):
        return kda.kda_pages(base, page, stride, layers, slots)

    def copy(pg, n=2, src=D):
        return lib.kda_pool_copy(pg, src, D, n, None, None)

    assert copy(pages(base=None)) == copy(pages(), src=None) == kda.KDA_ERR_NULL_ARG
    assert copy(pages(slots=0)) == copy(pages(page=0)) == copy(pages(), n=-1) == kda.KDA_ERR_SHAPE
    assert copy(pages(stride=8176)) == kda.KDA_ERR_SHAPE  # the layers would overlap
    assert copy(pages(page=1000)) == copy(pages(base=0x10008)) == copy(pages(stride=8200)) == kda.KDA_ERR_ALIGNMENT
    assert copy(pages(slots=(1 << 19) + 1, layers=1)) == kda.KDA_ERR_UNSUPPORTED
    assert copy(pages(), n=0) == kda.KDA_OK
    assert lib.kda_pool_free(None, 8, D, 4, D, 2, None, None) == kda.KDA_ERR_NULL_ARG
    assert lib.kda_pool_free(ODD, 8, D, 4, D, 2, None, None) == kda.KDA_ERR_ALIGNMENT
    assert lib.kda_pool_free(D, 0, D, 4, D, 2, None, None) == kda.KDA_ERR_SHAPE
    assert lib.kda_pool_compact(pages(), D, D, 4, None, None, None) == kda.KDA_ERR_NULL_ARG
    assert lib.kda_pool_compact(pages(), ODD, D, 4, D, None, None) == kda.KDA_ERR_ALIGNMENT
    assert lib.kda_pool_compact(pages(), D, D, -1, D, None, None) == kda.KDA_ERR_SHAPE
    assert lib.kda_pool_fork(pages(), D, D, 4, None, D, 2, D, None, None) == kda.KDA_ERR_NULL_ARG
    assert lib.kda_pool_fork(pages(), D, D, 4, D, D, -1, D, None, None) == kda.KDA_ERR_SHAPE
    assert lib.kda_pool_fork(pages(), D, D, 4, D, D, 2, None, None, None) == kda.KDA_ERR_NULL_ARG


def test_binding_refuses_wrong_shapes_and_types():
    bf, i32 = torch.bfloat16, torch.int32
    d = kda.dims(1, HV=2)
    x = dict(q=torch.zeros(4, 1, 128, dtype=bf), k=torch.zeros(4, 1, 128, dtype=bf), v=torch.zeros(4, 2, 128, dtype=bf),
             a=torch.zeros(4, 2, dtype=bf), b=torch.zeros(4, 2, dtype=bf), state_pool=torch.zeros(3, 2, 128, 128),
             state_idx=torch.zeros(1, dtype=i32), cu_seqlens=torch.zeros(2, dtype=i32), num_seqs=1,
             o=torch.zeros(4, 2, 128, dtype=bf))

    def call(**kw):
        kda.kda_gdn_prefill(d, kda.ScalarGate(), **{**x, "a": x["a"].float(), **kw})

    with pytest.raises(ValueError, match="device tensors"):
        call()
    for bad in (dict(a=torch.zeros(4, 3)), dict(o=x["o"][:3]), dict(v=x["v"][:, :1]), dict(b=x["b"][:3]),
                dict(state_pool=torch.zeros(3, 1, 128, 128)), dict(cu_seqlens=torch.zeros(1, dtype=i32)),
                dict(intermediate=torch.zeros(2, 1, 128, 128))):
        with pytest.raises(ValueError):
            call(**bad)
    p, tok = torch.rand(2, 3, 10), torch.zeros(2, 3, dtype=i32)
    u, out = torch.rand(2, 3), torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="device tensors"):
        kda.kda_accept_chain(p, p[:, :2].contiguous(), tok, u, out, out)
    with pytest.raises(ValueError):  # the rows of a slice do not lie one stride apart
        kda.kda_accept_chain(p, p[:, :2], tok, u, out, out)
    with pytest.raises(ValueError):
        kda.kda_accept_chain(p, p[:, :2, :9].contiguous(), tok, u, out, out)
    with pytest.raises(ValueError):
        kda.kda_accept_chain(p[:, :2], None, tok, u, out, out)
    with pytest.raises(TypeError):
        kda.kda_accept_chain(p.double(), None, tok, u, out, out)
    with pytest.raises(ValueError):
        kda.kda_accept_tree(p, tok, tok, u, out, out, out)  # path [B, T]
    with pytest.raises(ValueError):
        kda.kda_pool_copy(torch.zeros(2, 8, 16).transpose(1, 2), out, out)
    with pytest.raises(ValueError):
        kda.kda_pool_copy(torch.zeros(2, 8, 16), out, out[:1])
    with pytest.raises(TypeError):
        kda.kda_pool_free(torch.zeros(8), out, out)


def test_oracle_invariants():
    rng = np.random.default_rng(0)
    S = rng.normal(size=(2, 3, 4))
    q, k, v = rng.normal(size=(1, 4)), rng.normal(size=(1, 4)), rng.normal(size=(2, 3))
    unit = k / np.sqrt((k * k).sum() + 1e-6)
    # no decay, beta 1, unit key: the new state reads v at k; beta 0: unchanged
    S1, o = so.gdn_step(S, q, k / np.linalg.norm(k), v, np.ones(2), np.ones(2), 1.0, l2norm=False)
    assert np.allclose(np.einsum("hvk,k->hv", S1, k[0] / np.linalg.norm(k)), v)
    assert np.array_equal(so.gdn_step(S, q, k, v, np.ones(2), np.zeros(2), 1.0)[0], S)
    # the rule as written with a matrix
    al, be = np.array([0.7, 0.9]), np.array([0.3, 0.8])
    S2, _ = so.gdn_step(S, q, k, v, al, be, 1.0)
    for h in range(2):
        kk = unit[0]
        want = (np.eye(4) - be[h] * np.outer(kk, kk)) @ (al[h] * S[h].T) + be[h] * np.outer(kk, v[h])
        assert np.allclose(S2[h], want.T)
    # accepted tokens are distributed as the target, whatever proposed them
    p, qd = np.array([[0.5, 0.3, 0.2], [0.2, 0.2, 0.6]]), np.array([[0.2, 0.2, 0.6]])
    got = np.zeros(3)
    for _ in range(20000):
        t = rng.choice(3, p=qd[0])
        a, n = so.accept_chain(p, qd, [0, t], rng.random(2), 2)
        got[t if a == 1 else n] += 1
    assert np.abs(got / got.sum() - p[0]).max() < 4 * 0.5 / np.sqrt(20000)
    got[:] = 0
    for _ in range(20000):
        a, _, n = so.accept_tree(p[[0, 1, 1]], [0, 2, 0], [-1, 0, 0], rng.random(3), 3)
        got[[n, 2, 0][a]] += 1
    assert np.abs(got / got.sum() - p[0]).max() < 4 * 0.5 / np.sqrt(20000)
