"""Refusals, without a GPU, of linear attention, token log probabilities and the
archive of pages: host status codes of the C ABI (every call returns before it
touches the device) and the binding's rules; and the oracle's invariants."""
import ctypes

import numpy as np
import pytest
import torch

from linear_attention_serving_gated_gb300 import build, kda
from oracle import serving_oracle as so

D = ctypes.c_void_p(0x10000)  # never dereferenced
ODD = ctypes.c_void_p(0x10002)
bf, i32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kda.load()


def sgate(A_log=D):
    return kda.kda_scalar_gate(A_log, None, 1, 1, 128 ** -0.5)


def test_lin_host_errors(lib):
    row = 3 * 16 * 128

    def pre(d=kda.dims(16), g=sgate(), q=D, a=D, pool=D, idx=D, rows=64, T=64, n=1, o=D, ws=D, ws_bytes=1 << 40):
        return lib.kda_lin_prefill(d, g, q, D, D, a, rows, pool, 4, idx, None, n, T, o, ws, ws_bytes, None, None)

    assert pre(pool=None) == pre(idx=None) == pre(q=None) == pre(o=None) == kda.KDA_ERR_NULL_ARG
    assert pre(a=None, g=sgate(None)) == kda.KDA_ERR_NULL_ARG  # nothing to decay by
    assert pre(rows=63) == pre(T=65, rows=65, n=2) == pre(T=2 ** 31, rows=2 ** 31) == pre(n=0) == pre(n=-1) == kda.KDA_ERR_SHAPE
    assert pre(d=kda.dims(4, K=64, V=64)) == pre(d=kda.dims(4, HV=6)) == pre(d=kda.dims(4, dtype=2)) == kda.KDA_ERR_UNSUPPORTED
    assert pre(q=ODD) == pre(pool=ODD) == pre(o=ODD) == kda.KDA_ERR_ALIGNMENT
    assert pre(g=sgate(None), a=ODD) == pre(a=ctypes.c_void_p(0x10001)) == kda.KDA_ERR_ALIGNMENT
    assert pre(T=0, rows=0) == kda.KDA_OK  # nothing to do
    assert kda.kda_lin_prefill_workspace_size(kda.dims(16), 1, 2 ** 31) == 2 ** 64 - 1
    need = kda.kda_lin_prefill_workspace_size(kda.dims(16), 1, 4096)
    assert need > 0 == kda.kda_lin_prefill_workspace_size(kda.dims(16), 1, 64)
    assert pre(T=4096, rows=4096, ws=None) == pre(T=4096, rows=4096, ws_bytes=need - 1) == kda.KDA_ERR_WORKSPACE
    assert pre(T=4096, rows=4096, ws=ODD) == kda.KDA_ERR_ALIGNMENT

    def dec(d=kda.dims(16), g=sgate(), stride=row, a=D, pool=D, qkv=D, B=2):
        return lib.kda_lin_decode_packed(d, g, qkv, stride, a, B, pool, 240, D, D, None, None)

    assert dec(pool=None) == dec(qkv=None) == dec(g=sgate(None), a=None) == kda.KDA_ERR_NULL_ARG
    assert dec(stride=row - 8) == dec(B=-1) == kda.KDA_ERR_SHAPE
    assert dec(stride=row + 4) == dec(qkv=ODD) == kda.KDA_ERR_ALIGNMENT
    assert dec(d=kda.dims(16, HV=24)) == kda.KDA_ERR_UNSUPPORTED
    assert dec(B=0) == kda.KDA_OK
    d = kda.dims(16)
    assert lib.kda_lin_verify_chain(d, sgate(), D, row, D, 2, 0, D, 9, D, D, D, None, None) == kda.KDA_ERR_SHAPE
    assert lib.kda_lin_verify_chain(d, sgate(), D, row, D, 2, 6, D, 9, D, D, None, None, None) == kda.KDA_ERR_NULL_ARG
    assert lib.kda_lin_verify_tree(d, sgate(), D, row, D, 2, 6, None, D, 9, D, D, D, None, None) == kda.KDA_ERR_NULL_ARG
    assert lib.kda_lin_verify_chain(d, sgate(), D, row, D, 2, 6, D, 9, D, D, ODD, None, None) == kda.KDA_ERR_ALIGNMENT


def test_logprobs_host_errors(lib):
    def call(dt=2, x=D, stride=100, tokens=D, rows=2, V=100, lp=D, top=0, tt=D, tl=D):
        return lib.kda_token_logprobs(dt, x, stride, tokens, rows, V, lp, None, top, tt, tl, None, None)

    assert call(dt=3) == call(dt=-1) == call(top=33) == call(V=(1 << 28) + 1, stride=1 << 30) == kda.KDA_ERR_UNSUPPORTED
    assert call(x=None) == call(tokens=None) == call(lp=None) == call(top=1, tt=None) == call(top=1, tl=None) == kda.KDA_ERR_NULL_ARG
    assert call(stride=99) == call(V=0) == call(rows=-1) == call(top=-1) == kda.KDA_ERR_SHAPE
    assert call(x=ODD) == call(dt=0, x=ctypes.c_void_p(0x10001)) == kda.KDA_ERR_ALIGNMENT
    assert call(rows=0) == kda.KDA_OK


def test_archive_host_errors(lib):
    def call(name="kda_pool_store", base=0x10000, page=1024, stride=8192, layers=2, slots=8, codes=0x10000, scales=0x10000, bits=8,
             keep=4, src=D, n=2):
        return getattr(lib, name)(kda.kda_pages(base, page, stride, layers, slots), kda.kda_archive(codes, scales, bits, keep), src, D,
                                  n, None, None)

    for name in ("kda_pool_store", "kda_pool_load"):
        c = lambda **kw: call(name, **kw)  # noqa: E731
        assert c(base=None) == c(codes=None) == c(scales=None) == c(src=None) == kda.KDA_ERR_NULL_ARG
        assert c(slots=0) == c(page=0) == c(layers=0) == c(keep=0) == c(n=-1) == c(stride=8176) == kda.KDA_ERR_SHAPE
        assert c(bits=2) == c(page=1040, stride=8320) == kda.KDA_ERR_UNSUPPORTED
        assert c(base=0x10008) == c(stride=8200) == c(codes=0x10004) == c(scales=0x10004) == kda.KDA_ERR_ALIGNMENT
        assert c(n=0) == kda.KDA_OK
        assert c(page=1 << 40, stride=1 << 60, n=2 ** 20) == kda.KDA_ERR_SHAPE  # more CTAs than a grid has


def test_binding_refuses_wrong_shapes_and_types():
    d = kda.dims(1, HV=2)
    x = dict(q=torch.zeros(4, 1, 128, dtype=bf), k=torch.zeros(4, 1, 128, dtype=bf), v=torch.zeros(4, 2, 128, dtype=bf),
             a=torch.zeros(4, 2), state_pool=torch.zeros(3, 2, 128, 128), state_idx=torch.zeros(1, dtype=i32),
             cu_seqlens=torch.zeros(2, dtype=i32), num_seqs=1, o=torch.zeros(4, 2, 128, dtype=bf))

    def call(**kw):
        kda.kda_lin_prefill(d, kda.ScalarGate(), **{**x, **kw})

    with pytest.raises(ValueError, match="device tensors"):
        call()
    for bad in (dict(a=torch.zeros(4, 3)), dict(o=x["o"][:3]), dict(v=x["v"][:, :1]), dict(state_pool=torch.zeros(3, 1, 128, 128)),
                dict(cu_seqlens=torch.zeros(1, dtype=i32)), dict(q=torch.zeros(4, 1, 256, dtype=bf)[..., ::2])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q=torch.zeros(4, 1, 128)), dict(a=torch.zeros(4, 2, dtype=bf)), dict(state_idx=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    rows = torch.zeros(2, 4 * 128, dtype=bf)
    with pytest.raises(ValueError):
        kda.kda_lin_decode_packed(d, kda.ScalarGate(), rows[:, :500], x["a"], x["state_pool"], x["state_idx"], x["o"])
    p, tok, out = torch.rand(3, 10), torch.zeros(3, dtype=i32), torch.zeros(3)
    with pytest.raises(ValueError, match="device tensors"):
        kda.kda_token_logprobs(p, tok, out)
    for bad in ((p[:2], tok, out), (p.T, torch.zeros(10, dtype=i32), torch.zeros(10)), (p[0], tok, out)):
        with pytest.raises(ValueError):
            kda.kda_token_logprobs(*bad)
    with pytest.raises(TypeError):
        kda.kda_token_logprobs(p.double(), tok, out)
    pool, codes, scales = torch.zeros(2, 4, 3, 128), torch.zeros(5, 2, 3, 128, dtype=torch.int8), torch.zeros(5, 2, 3)
    two = torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="device tensors"):
        kda.kda_pool_store(pool, codes, scales, two, two)
    with pytest.raises(TypeError):
        kda.kda_pool_store(pool, codes.float(), scales, two, two)
    with pytest.raises(ValueError):
        kda.kda_pool_load(codes, scales, pool, two, two[:1])


def test_oracle_invariants():
    rng = np.random.default_rng(0)
    T, H, HV, K, V = 12, 2, 4, 5, 3
    q, k, v = rng.normal(size=(T, H, K)), rng.normal(size=(T, H, K)), rng.normal(size=(T, HV, V))
    S0, g = rng.normal(size=(HV, V, K)), -rng.random((T, HV))
    o, states = so.lin_sequence(S0, q, k, v, g, 0.7, l2norm=False)
    # the attention written as a sum over the tokens before
    c = np.cumsum(g, 0)
    for h in range(HV):
        w = np.tril(np.exp(c[:, None, h] - c[None, :, h])) * (q[:, h // 2] @ k[:, h // 2].T)
        want = w @ v[:, h] + np.exp(c[:, h])[:, None] * (q[:, h // 2] @ S0[h].T)
        assert np.allclose(o[:, h], 0.7 * want)
    assert np.allclose(states[3], so.lin_sequence(S0, q[:4], k[:4], v[:4], g[:4], 1.0, l2norm=False)[1][-1])
    # the gated delta rule without its correction: beta v against a state that gives nothing at k
    assert np.allclose(so.lin_decay(3, None, np.zeros(2)), -1)
    assert np.allclose(so.lin_decay(1, [[3.0, -500.0]]), [[0, -128]])
    lp, ent, tok, lps = so.logprobs([1.0, 1.0, -np.inf, 3.0], 1, 4)
    p = np.exp([1.0, 1.0, 3.0])
    p /= p.sum()
    assert np.isclose(lp, np.log(p[1])) and np.isclose(ent, -(p * np.log(p)).sum()) and tok.tolist() == [3, 0, 1, -1]
    assert so.logprobs([-np.inf] * 3, 0, 1)[0] == -np.inf
    x = np.concatenate([np.arange(-127, 1), np.arange(128)]).reshape(2, 128).astype(np.float32)
    codes, scales, value = so.archived(x, 8)
    assert np.array_equal(codes, x) and (scales == 1).all() and np.array_equal(value, x)
    assert np.abs(so.archived(x, 4)[2] - x).max() <= 127 / 14 + 1e-5
