"""ctypes binding of libkda (include/kda.h): the same entry points, taking
torch tensors on the GPU and marshalling them to device pointers.

Every step of the computation runs in the library's CUDA kernels; this
module only checks dtypes/devices, passes pointers, sizes and the current
stream, and raises ``KdaError`` on a non-OK status.  If ``libkda.so`` is
missing it raises at the first call: there is no other implementation.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from . import build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")

KDA_OK = 0
KDA_ERR_NULL_ARG = 1
KDA_ERR_SHAPE = 2
KDA_ERR_UNSUPPORTED = 3
KDA_ERR_WORKSPACE = 4
KDA_ERR_CUDA = 5
KDA_ERR_ALIGNMENT = 6

KDA_DEVERR_SLOT = 1
KDA_DEVERR_PARENT = 2
KDA_DEVERR_SEQLENS = 4
KDA_DEVERR_ACCEPTED = 8
KDA_DEVERR_TIMEOUT = 16
KDA_DEVERR_INTERMEDIATE = 32
KDA_DEVERR_TOKEN = 64
KDA_DEVERR_PAGE = 128
KDA_DEVERR_POOL_FULL = 256

CHUNK = 64


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


KDA_DTYPE_BF16, KDA_DTYPE_F16 = 0, 1
KDA_DTYPE_F32 = 2  # probabilities of kda_accept_chain / kda_accept_tree only


class kda_dims(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("HV", ctypes.c_int), ("K", ctypes.c_int), ("V", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class kda_gate(ctypes.Structure):
    _fields_ = [("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("lower_bound", ctypes.c_float), ("beta_is_raw", ctypes.c_int),
                ("use_qk_l2norm", ctypes.c_int), ("scale", ctypes.c_float)]


class kda_scalar_gate(ctypes.Structure):
    _fields_ = [("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p), ("beta_is_raw", ctypes.c_int),
                ("use_qk_l2norm", ctypes.c_int), ("scale", ctypes.c_float)]


class kda_pages(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
                ("layers", ctypes.c_int), ("slots", ctypes.c_int)]


class kda_archive(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("bits", ctypes.c_int), ("slots", ctypes.c_int)]


EXPORTS = ("kda_status_string", "kda_prefill_workspace_size", "kda_prefill", "kda_decode_packed",
           "kda_verify_chain", "kda_verify_tree", "kda_commit", "kda_set_stage_events",
           "kda_prefill_noalloc", "kda_replay_ring_bytes", "kda_verify_chain_replay",
           "kda_commit_replay", "kda_gdn_prefill_workspace_size", "kda_gdn_prefill", "kda_gdn_decode_packed", "kda_gdn_verify_chain",
           "kda_gdn_verify_tree", "kda_accept_chain", "kda_accept_tree", "kda_pool_copy", "kda_pool_free",
           "kda_pool_compact", "kda_pool_fork", "kda_lin_prefill_workspace_size", "kda_lin_prefill",
           "kda_lin_decode_packed", "kda_lin_verify_chain", "kda_lin_verify_tree", "kda_token_logprobs",
           "kda_pool_store", "kda_pool_load")

PREFILL_STATIC_SCRATCH_BYTES = 128 << 20  # KDA_PREFILL_STATIC_SCRATCH_BYTES in include/kda.h

_lib = None


def load(path: str = LIB_PATH):
    """Load libkda.so (built by build.py).  Raises if it is missing."""
    global _lib, _arg, _rows, _states, _place
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"libkda.so not built ({path}); run linear_attention_serving_gated_gb300.build.build()")
        built, here = build.built_for(), build.made_for()
        if built is not None and built != here:  # it would read tensors by another layout
            raise RuntimeError(f"_host_args.so is built for {built}; this is {here}: run "
                               "linear_attention_serving_gated_gb300.build.build()")
        try:
            if built is None:
                raise ImportError("what it is built for is not known")
            from . import _host_args  # built beside it
        except ImportError as e:
            raise RuntimeError("_host_args.so not built; run linear_attention_serving_gated_gb300.build.build()") from e
        _host_args.otherwise(_checked_arg)
        _arg, _rows, _states, _place = _host_args.arg, _host_args.rows, _host_args.states, _host_args.place
        lib = ctypes.CDLL(path)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_status_string.argtypes = [i32]
        lib.kda_prefill_workspace_size.restype = sz
        lib.kda_prefill_workspace_size.argtypes = [kda_dims, i32, i64]
        lib.kda_prefill.restype = i32
        lib.kda_prefill.argtypes = [kda_dims, kda_gate, vp, vp, vp, vp, vp, i64, vp, i32, vp, vp, i32,
                                    i64, vp, vp, i64, vp, sz, vp, vp]
        lib.kda_decode_packed.restype = i32
        lib.kda_decode_packed.argtypes = [kda_dims, kda_gate, vp, i64, vp, vp, i32, vp, i32, vp, vp,
                                          vp, vp]
        lib.kda_verify_chain.restype = i32
        lib.kda_verify_chain.argtypes = [kda_dims, kda_gate, vp, i64, vp, vp, i32, i32, vp, i32, vp,
                                         vp, vp, vp, vp]
        lib.kda_verify_tree.restype = i32
        lib.kda_verify_tree.argtypes = [kda_dims, kda_gate, vp, i64, vp, vp, i32, i32, vp, vp, i32,
                                        vp, vp, vp, vp, vp]
        lib.kda_commit.restype = i32
        lib.kda_commit.argtypes = [kda_dims, vp, i32, i32, vp, vp, i32, vp, vp, vp]
        lib.kda_prefill_noalloc.restype = i32
        lib.kda_prefill_noalloc.argtypes = [kda_dims, kda_gate, vp, vp, vp, vp, vp, i64, vp, i32, vp,
                                            vp, i32, i64, vp, vp, i64, vp, vp]
        lib.kda_replay_ring_bytes.restype = sz
        lib.kda_replay_ring_bytes.argtypes = [kda_dims, i32, i32]
        lib.kda_verify_chain_replay.restype = i32
        lib.kda_verify_chain_replay.argtypes = [kda_dims, kda_gate, vp, i64, vp, vp, i32, i32, vp, i32,
                                                vp, vp, vp, vp, vp]
        lib.kda_commit_replay.restype = i32
        lib.kda_commit_replay.argtypes = [kda_dims, vp, i32, i32, vp, vp, i32, vp, vp, vp]
        lib.kda_gdn_prefill.restype = i32
        lib.kda_gdn_prefill_workspace_size.restype = sz
        lib.kda_gdn_prefill_workspace_size.argtypes = [kda_dims, i32, i64]
        lib.kda_gdn_prefill.argtypes = [kda_dims, kda_scalar_gate, vp, vp, vp, vp, vp, i64, vp, i32, vp, vp,
                                        i32, i64, vp, vp, i64, vp, sz, vp, vp]
        lib.kda_gdn_decode_packed.restype = i32
        lib.kda_gdn_decode_packed.argtypes = [kda_dims, kda_scalar_gate, vp, i64, vp, vp, i32, vp, i32, vp,
                                              vp, vp, vp]
        lib.kda_gdn_verify_chain.restype = i32
        lib.kda_gdn_verify_chain.argtypes = [kda_dims, kda_scalar_gate, vp, i64, vp, vp, i32, i32, vp, i32,
                                             vp, vp, vp, vp, vp]
        lib.kda_gdn_verify_tree.restype = i32
        lib.kda_gdn_verify_tree.argtypes = [kda_dims, kda_scalar_gate, vp, i64, vp, vp, i32, i32, vp, vp,
                                            i32, vp, vp, vp, vp, vp]
        lib.kda_accept_chain.restype = i32
        lib.kda_accept_chain.argtypes = [i32, vp, i64, vp, i64, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp]
        lib.kda_accept_tree.restype = i32
        lib.kda_accept_tree.argtypes = [i32, vp, i64, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp]
        lib.kda_pool_copy.restype = i32
        lib.kda_pool_copy.argtypes = [kda_pages, vp, vp, i32, vp, vp]
        lib.kda_pool_free.restype = i32
        lib.kda_pool_free.argtypes = [vp, i32, vp, i32, vp, i32, vp, vp]
        lib.kda_pool_compact.restype = i32
        lib.kda_pool_compact.argtypes = [kda_pages, vp, vp, i32, vp, vp, vp]
        lib.kda_pool_fork.restype = i32
        lib.kda_pool_fork.argtypes = [kda_pages, vp, vp, i32, vp, vp, i32, vp, vp, vp]
        lib.kda_lin_prefill_workspace_size.restype = sz
        lib.kda_lin_prefill_workspace_size.argtypes = [kda_dims, i32, i64]
        lib.kda_lin_prefill.restype = i32
        lib.kda_lin_prefill.argtypes = [kda_dims, kda_scalar_gate, vp, vp, vp, vp, i64, vp, i32, vp, vp, i32, i64, vp,
                                        vp, sz, vp, vp]
        lib.kda_lin_decode_packed.restype = i32
        lib.kda_lin_decode_packed.argtypes = [kda_dims, kda_scalar_gate, vp, i64, vp, i32, vp, i32, vp, vp, vp, vp]
        lib.kda_lin_verify_chain.restype = i32
        lib.kda_lin_verify_chain.argtypes = [kda_dims, kda_scalar_gate, vp, i64, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp]
        lib.kda_lin_verify_tree.restype = i32
        lib.kda_lin_verify_tree.argtypes = [kda_dims, kda_scalar_gate, vp, i64, vp, i32, i32, vp, vp, i32, vp, vp, vp, vp,
                                            vp]
        lib.kda_token_logprobs.restype = i32
        lib.kda_token_logprobs.argtypes = [i32, vp, i64, vp, i32, i32, vp, vp, i32, vp, vp, vp, vp]
        for call in (lib.kda_pool_store, lib.kda_pool_load):
            call.restype = i32
            call.argtypes = [kda_pages, kda_archive, vp, vp, i32, vp, vp]
        lib.kda_set_stage_events.restype = None
        lib.kda_set_stage_events.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    try:
        return load().kda_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def _check(status: int, where: str):
    if status != KDA_OK:
        raise KdaError(status, where)


def _p(t):
    """Device pointer of a tensor (or None)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libkda takes device tensors")
    return ctypes.c_void_p(t.data_ptr())


def _in16(d, t, name):
    """A 16-bit token tensor: bfloat16 (or float16 when d.dtype is F16); int16
    raw bits are accepted either way."""
    want = torch.float16 if d.dtype == KDA_DTYPE_F16 else torch.bfloat16
    if t is not None and t.dtype not in (want, torch.int16):
        raise TypeError(f"{name} must be {want} (got {t.dtype})")
    return _p(t)


def _at_least(t, n, name, shape):
    """t must be dense (the library indexes it by its documented layout) and
    hold n elements (the rows the kernels touch); t None allowed."""
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < n:
        raise ValueError(f"{name} must hold {shape} = {n} elements (got shape {tuple(t.shape)})")


def _packed_shapes(d, mixed_qkv, a, b, state_pool, state_idx, rows, reqs):
    """Shape rules of a packed-row call, checked on the host because the
    library sees only pointers.  As the pages' packed-decode validator does
    ("PR #35197 report: fix(kernel) Fix Helion small-token prefill bug",
    kda_decode.py snippet), HV, V and K come from the state's trailing
    dimensions and the gate input `a` must be [rows, HV*K]; every row the
    kernels read (rows = requests x tokens) must exist."""
    if state_pool.dim() < 3 or tuple(state_pool.shape[-3:]) != (d.HV, d.V, d.K):
        raise ValueError(f"state_pool must end in [HV, V, K] = [{d.HV}, {d.V}, {d.K}] "
                         f"(got {tuple(state_pool.shape)})")
    _at_least(state_pool, 0, "state_pool", "[slots, HV, V, K]")
    width = 2 * d.H * d.K + d.HV * d.V
    if mixed_qkv.dim() != 2 or mixed_qkv.shape[0] < rows or mixed_qkv.shape[1] < width \
            or mixed_qkv.stride(1) != 1:
        raise ValueError(f"mixed_qkv must be [>= {rows}, >= {width}] with unit column stride "
                         f"(got {tuple(mixed_qkv.shape)})")
    if a.shape[-1] != d.HV * d.K or a.numel() < rows * d.HV * d.K or not a.is_contiguous():
        raise ValueError(f"`a` must have shape [B, HV*K] = [{rows}, {d.HV * d.K}], contiguous "
                         f"(got {tuple(a.shape)})")
    if b.numel() < rows * d.HV or not b.is_contiguous():
        raise ValueError(f"`b` must have shape [B, HV] = [{rows}, {d.HV}], contiguous "
                         f"(got {tuple(b.shape)})")
    _at_least(state_idx, reqs, "state_idx", f"[{reqs}]")


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class Gate:
    """Fold options of a call (kda_gate): A_log [HV] / dt_bias [HV*K] FP32
    device tensors or None, lower_bound (None = unbounded, rejected when
    A_log is given), beta_is_raw, use_qk_l2norm, scale."""

    def __init__(self, A_log=None, dt_bias=None, lower_bound=-5.0, beta_is_raw=True,
                 use_qk_l2norm=True, scale=128 ** -0.5):
        self.A_log, self.dt_bias = A_log, dt_bias
        self.lower_bound = lower_bound
        self.beta_is_raw, self.use_qk_l2norm, self.scale = beta_is_raw, use_qk_l2norm, scale

    def c(self):
        for t in (self.A_log, self.dt_bias):
            if t is not None and t.dtype != torch.float32:
                raise TypeError("A_log and dt_bias must be float32")
        lb = float("nan") if self.lower_bound is None else float(self.lower_bound)
        return kda_gate(_p(self.A_log), _p(self.dt_bias), lb, int(bool(self.beta_is_raw)),
                        int(bool(self.use_qk_l2norm)), float(self.scale))


def dims(H, K=128, V=128, HV=None, dtype=KDA_DTYPE_BF16):
    """Head counts and sizes of a call; dtype: element type of the 16-bit
    token tensors and of o (KDA_DTYPE_BF16 or KDA_DTYPE_F16)."""
    return kda_dims(int(H), int(HV if HV is not None else H), int(K), int(V), int(dtype))


def kda_prefill_workspace_size(d: kda_dims, num_seqs: int, total_tokens: int) -> int:
    return int(load().kda_prefill_workspace_size(d, int(num_seqs), int(total_tokens)))


def _intermediate_chunks(d, intermediate):
    """Chunk records an intermediate-state buffer holds: it must be a dense
    [chunks, HV, V, K] FP32 tensor.  The library writes only that many (the
    chunk count follows cu_seqlens, which is on the device) and flags the
    rest."""
    if intermediate is None:
        return 0
    if intermediate.dtype != torch.float32 or intermediate.dim() != 4 or \
            tuple(intermediate.shape[1:]) != (d.HV, d.V, d.K):
        raise ValueError(f"intermediate must be float32 [chunks, HV, V, K] = [*, {d.HV}, {d.V}, {d.K}] "
                         f"(got {intermediate.dtype} {tuple(intermediate.shape)})")
    _at_least(intermediate, 0, "intermediate", "[chunks, HV, V, K]")
    return int(intermediate.shape[0])


def _space(workspace):
    """(device pointer, bytes) of a workspace: dense, so that it holds its bytes at its pointer."""
    _at_least(workspace, 0, "workspace", "[bytes]")
    return _here(workspace), workspace.numel() * workspace.element_size()


def _prefill_shapes(d, q, k, v, g, beta, state_pool, state_idx, cu_seqlens, num_seqs, o):
    """Every element the prefill kernels touch for T = q.shape[0] tokens and
    gb_rows = g.shape[0] gate rows must exist (the library sees pointers)."""
    T, gb_rows, n = q.shape[0], g.shape[0], int(num_seqs)
    if state_pool.dim() < 3 or tuple(state_pool.shape[-3:]) != (d.HV, d.V, d.K):
        raise ValueError(f"state_pool must end in [HV, V, K] = [{d.HV}, {d.V}, {d.K}] "
                         f"(got {tuple(state_pool.shape)})")
    _at_least(state_pool, 0, "state_pool", "[slots, HV, V, K]")
    _at_least(q, T * d.H * d.K, "q", f"[{T}, H, K]")
    _at_least(k, T * d.H * d.K, "k", f"[{T}, H, K]")
    _at_least(v, T * d.HV * d.V, "v", f"[{T}, HV, V]")
    _at_least(g, gb_rows * d.HV * d.K, "g", f"[{gb_rows}, HV, K]")
    _at_least(beta, gb_rows * d.HV, "beta", f"[{gb_rows}, HV]")
    _at_least(o, T * d.HV * d.V, "o", f"[{T}, HV, V]")
    _at_least(state_idx, n, "state_idx", f"[{n}]")
    _at_least(cu_seqlens, n + 1, "cu_seqlens", f"[{n + 1}]")


def kda_prefill(d, gate: Gate, q, k, v, g, beta, state_pool, state_idx, cu_seqlens, num_seqs,
                o, intermediate=None, workspace=None, err_flag=None, stream=None):
    """Chunked varlen prefill (see kda.h).  q,k [T,H,K], v [T,HV,V], g
    [gb_rows,HV,K], beta [gb_rows,HV] bf16; state_pool [slots,HV,V,K] fp32
    (in place); o [T,HV,V] bf16 (written)."""
    T = q.shape[0]
    gb_rows = g.shape[0]
    _prefill_shapes(d, q, k, v, g, beta, state_pool, state_idx, cu_seqlens, num_seqs, o)
    inter_chunks = _intermediate_chunks(d, intermediate)
    if workspace is None:
        need = kda_prefill_workspace_size(d, num_seqs, T)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = load().kda_prefill(
        d, gate.c(), _in16(d, q, "q"), _in16(d, k, "k"), _in16(d, v, "v"), _in16(d, g, "g"), _in16(d, beta, "beta"),
        int(gb_rows), _p(state_pool), int(state_pool.shape[0]), _p(state_idx), _p(cu_seqlens),
        int(num_seqs), int(T), _in16(d, o, "o"), _p(intermediate), inter_chunks, *_space(workspace),
        _p(err_flag), _stream(stream))
    _check(st, "kda_prefill")


def kda_prefill_noalloc(d, gate: Gate, q, k, v, g, beta, state_pool, state_idx, cu_seqlens,
                        num_seqs, o, intermediate=None, err_flag=None, stream=None):
    """kda_prefill with the library's built-in static scratch (see kda.h): for
    callers that cannot allocate device memory."""
    _prefill_shapes(d, q, k, v, g, beta, state_pool, state_idx, cu_seqlens, num_seqs, o)
    inter_chunks = _intermediate_chunks(d, intermediate)
    st = load().kda_prefill_noalloc(
        d, gate.c(), _in16(d, q, "q"), _in16(d, k, "k"), _in16(d, v, "v"), _in16(d, g, "g"), _in16(d, beta, "beta"),
        int(g.shape[0]), _p(state_pool), int(state_pool.shape[0]), _p(state_idx), _p(cu_seqlens),
        int(num_seqs), int(q.shape[0]), _in16(d, o, "o"), _p(intermediate), inter_chunks,
        _p(err_flag), _stream(stream))
    _check(st, "kda_prefill_noalloc")


def kda_decode_packed(d, gate: Gate, mixed_qkv, a, b, state_pool, state_idx, o, err_flag=None,
                      stream=None):
    B = mixed_qkv.shape[0]
    _packed_shapes(d, mixed_qkv, a, b, state_pool, state_idx, B, B)
    _at_least(o, B * d.HV * d.V, "o", f"[{B}, HV, V]")
    st = load().kda_decode_packed(
        d, gate.c(), _in16(d, mixed_qkv, "mixed_qkv"), int(mixed_qkv.stride(0)), _in16(d, a, "a"),
        _in16(d, b, "b"), int(mixed_qkv.shape[0]), _p(state_pool), int(state_pool.shape[0]),
        _p(state_idx), _in16(d, o, "o"), _p(err_flag), _stream(stream))
    _check(st, "kda_decode_packed")


def _verify_shapes(d, mixed_qkv, a, b, B, T, state_pool, state_idx, o):
    rows = int(B) * int(T)
    _packed_shapes(d, mixed_qkv, a, b, state_pool, state_idx, rows, int(B))
    _at_least(o, rows * d.HV * d.V, "o", f"[{B}, {T}, HV, V]")


def kda_verify_chain(d, gate: Gate, mixed_qkv, a, b, B, T, state_pool, state_idx, o, snapshots,
                     err_flag=None, stream=None):
    _verify_shapes(d, mixed_qkv, a, b, B, T, state_pool, state_idx, o)
    _at_least(snapshots, B * T * d.HV * d.V * d.K, "snapshots", f"[{B}, {T}, HV, V, K]")
    st = load().kda_verify_chain(
        d, gate.c(), _in16(d, mixed_qkv, "mixed_qkv"), int(mixed_qkv.stride(0)), _in16(d, a, "a"),
        _in16(d, b, "b"), int(B), int(T), _p(state_pool), int(state_pool.shape[0]), _p(state_idx),
        _in16(d, o, "o"), _p(snapshots), _p(err_flag), _stream(stream))
    _check(st, "kda_verify_chain")


def kda_verify_tree(d, gate: Gate, mixed_qkv, a, b, B, T, parent_idx, state_pool, state_idx, o,
                    snapshots, err_flag=None, stream=None):
    _verify_shapes(d, mixed_qkv, a, b, B, T, state_pool, state_idx, o)
    _at_least(snapshots, B * T * d.HV * d.V * d.K, "snapshots", f"[{B}, {T}, HV, V, K]")
    _at_least(parent_idx, B * T, "parent_idx", f"[{B}, {T}]")
    st = load().kda_verify_tree(
        d, gate.c(), _in16(d, mixed_qkv, "mixed_qkv"), int(mixed_qkv.stride(0)), _in16(d, a, "a"),
        _in16(d, b, "b"), int(B), int(T), _p(parent_idx), _p(state_pool), int(state_pool.shape[0]),
        _p(state_idx), _in16(d, o, "o"), _p(snapshots), _p(err_flag), _stream(stream))
    _check(st, "kda_verify_tree")


def kda_commit(d, snapshots, B, T, accepted, state_pool, state_idx, err_flag=None, stream=None):
    _at_least(snapshots, B * T * d.HV * d.V * d.K, "snapshots", f"[{B}, {T}, HV, V, K]")
    _at_least(accepted, B, "accepted", f"[{B}]")
    _at_least(state_idx, B, "state_idx", f"[{B}]")
    st = load().kda_commit(d, _p(snapshots), int(B), int(T), _p(accepted), _p(state_pool),
                           int(state_pool.shape[0]), _p(state_idx), _p(err_flag), _stream(stream))
    _check(st, "kda_commit")


def kda_replay_ring_bytes(d, B, T) -> int:
    return int(load().kda_replay_ring_bytes(d, int(B), int(T)))


def kda_verify_chain_replay(d, gate: Gate, mixed_qkv, a, b, B, T, state_pool, state_idx, o, ring,
                            err_flag=None, stream=None):
    """Chain verify without snapshots: o as kda_verify_chain, each token's
    folded inputs recorded in `ring` (kda_replay_ring_bytes bytes, FP32)."""
    _verify_shapes(d, mixed_qkv, a, b, B, T, state_pool, state_idx, o)
    _at_least(ring, kda_replay_ring_bytes(d, B, T) // 4, "ring", "kda_replay_ring_bytes / 4 FP32")
    st = load().kda_verify_chain_replay(
        d, gate.c(), _in16(d, mixed_qkv, "mixed_qkv"), int(mixed_qkv.stride(0)), _in16(d, a, "a"),
        _in16(d, b, "b"), int(B), int(T), _p(state_pool), int(state_pool.shape[0]), _p(state_idx),
        _in16(d, o, "o"), _p(ring), _p(err_flag), _stream(stream))
    _check(st, "kda_verify_chain_replay")


def kda_commit_replay(d, ring, B, T, accepted, state_pool, state_idx, err_flag=None, stream=None):
    """Advances each request's pool state through its accepted draft tokens
    from the ring written by kda_verify_chain_replay."""
    _at_least(ring, kda_replay_ring_bytes(d, B, T) // 4, "ring", "kda_replay_ring_bytes / 4 FP32")
    _at_least(accepted, B, "accepted", f"[{B}]")
    _at_least(state_idx, B, "state_idx", f"[{B}]")
    st = load().kda_commit_replay(d, _p(ring), int(B), int(T), _p(accepted), _p(state_pool),
                                  int(state_pool.shape[0]), _p(state_idx), _p(err_flag),
                                  _stream(stream))
    _check(st, "kda_commit_replay")


def kda_set_stage_events(events=None):
    """Profiling aid: torch.cuda.Event triple recorded by every later call
    (before its first kernel, between the prefill's two kernels, after its
    last kernel); a None entry is not recorded; None clears all three."""
    if events is None:
        load().kda_set_stage_events(None)
        return
    arr = (ctypes.c_void_p * 3)(*[ctypes.c_void_p(e.cuda_event if e is not None else None)
                                  for e in events])
    load().kda_set_stage_events(arr)


# -- the gated delta rule with one decay per value head ----------------------
#
# These calls take a few microseconds on the GPU at their smallest, so what the
# host does for one is kept short: one pass of checks per tensor, plain integers
# for pointers, and the current stream without a Python stream object.


def _here(t):
    """Device pointer of a tensor of the current device, on which the call runs."""
    at = _place(t)
    if at is not None:
        return at
    if not t.is_cuda:
        raise ValueError("libkda takes device tensors")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"libkda takes tensors of the current device, cuda:{torch._C._cuda_getDevice()} (got cuda:{t.get_device()})")
    return t.data_ptr()


def _checked_arg(t, dtype, n, name, shape):
    """Device pointer of a dense tensor of one element type that holds at least n
    elements (the rows the kernels touch), or what is wrong with it.  load() puts
    native code in front of it, as _arg."""
    if t.dtype is not dtype and not (t.dtype is torch.int16 and dtype in _BITS16):
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.numel() < n or not t.is_contiguous():
        _at_least(t, n, name, shape)
    return _here(t)


def _rows(t, dtype, n, width):
    """(device pointer, row stride) of at least n rows of `width` elements; None: not such
    a tensor (or load() has not put native code here yet)."""


def _states(t, HV, V, K):
    """(device pointer, slots) of a dense FP32 pool [slots, HV, V, K]; None as in _rows."""


def _place(t):
    """Device pointer of a tensor of the current device; None as in _rows."""


def _pool(d, t, HV, V, K):
    return _states(t, HV, V, K) or (_arg(t, torch.float32, 0, "state_pool", "[slots, HV, V, K]"), _pool_slots(d, t))


_arg = _checked_arg
_BITS16 = (torch.bfloat16, torch.float16)  # raw int16 bits are accepted for either


def _opt(t, dtype, n, name, shape):
    return None if t is None else _arg(t, dtype, n, name, shape)


def _err(err_flag):
    return None if err_flag is None else _arg(err_flag, torch.int32, 1, "err_flag", "[1]")


def _cur(stream):
    """cudaStream_t of a torch stream, or of the current one."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _new(n, dtype, device, stream):
    """Memory for a call's own use, of the allocator's pool for the stream it
    runs on: what another stream last used may still be in use there."""
    if stream is None:
        return torch.empty(n, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=dtype, device=device)


class ScalarGate:
    """Fold options of the kda_gdn_* calls (kda_scalar_gate): A_log and dt_bias
    [HV] FP32 device tensors.  Without A_log the gate input is the log-decay
    itself, FP32."""

    def __init__(self, A_log=None, dt_bias=None, beta_is_raw=True, use_qk_l2norm=True, scale=128 ** -0.5):
        self.A_log, self.dt_bias = A_log, dt_bias
        self.beta_is_raw, self.use_qk_l2norm, self.scale = beta_is_raw, use_qk_l2norm, scale

    def c(self, d):
        return kda_scalar_gate(_opt(self.A_log, torch.float32, d.HV, "A_log", "[HV]"),
                               _opt(self.dt_bias, torch.float32, d.HV, "dt_bias", "[HV]"),
                               1 if self.beta_is_raw else 0, 1 if self.use_qk_l2norm else 0, self.scale)


def _pool_slots(d, state_pool):
    shape = state_pool.shape
    if len(shape) != 4 or shape[1] != d.HV or shape[2] != d.V or shape[3] != d.K:
        raise ValueError(f"state_pool must be [slots, HV, V, K] = [*, {d.HV}, {d.V}, {d.K}] (got {tuple(shape)})")
    return shape[0]


def _gate_rows(d, gate, a, rows):
    """The gate input [>= rows, HV]: 16-bit with A_log, FP32 log-decays without."""
    if a.shape[-1] != d.HV:
        raise ValueError(f"`a` must have shape [rows, HV] = [{rows}, {d.HV}] (got {tuple(a.shape)})")
    return _arg(a, _t16(d) if gate.A_log is not None else torch.float32, rows * d.HV, "a", "[rows, HV]")


def _t16(d):
    return torch.float16 if d.dtype == KDA_DTYPE_F16 else torch.bfloat16


def kda_gdn_prefill_workspace_size(d: kda_dims, num_seqs: int, total_tokens: int) -> int:
    return int(load().kda_gdn_prefill_workspace_size(d, int(num_seqs), int(total_tokens)))


def kda_gdn_prefill(d, gate: ScalarGate, q, k, v, a, b, state_pool, state_idx, cu_seqlens, num_seqs, o,
                    intermediate=None, workspace=None, err_flag=None, stream=None):
    """Varlen prefill (see kda.h).  q,k [T,H,K], v [T,HV,V], a and b
    [gb_rows,HV]; state_pool [slots,HV,V,K] fp32 (in place); o [T,HV,V]
    (written)."""
    lib, t16 = load(), _t16(d)
    T, gb_rows, n = q.shape[0], a.shape[0], int(num_seqs)
    HK, HVV = d.H * d.K, d.HV * d.V
    slots = _pool_slots(d, state_pool)
    inter_chunks = _intermediate_chunks(d, intermediate) if intermediate is not None else 0
    if workspace is None:
        workspace = _new(max(int(lib.kda_gdn_prefill_workspace_size(d, n, T)), 1), torch.uint8, q.device, stream)
    st = lib.kda_gdn_prefill(
        d, gate.c(d), _arg(q, t16, T * HK, "q", "[T, H, K]"), _arg(k, t16, T * HK, "k", "[T, H, K]"),
        _arg(v, t16, T * HVV, "v", "[T, HV, V]"), _gate_rows(d, gate, a, gb_rows),
        _arg(b, t16, gb_rows * d.HV, "b", "[gb_rows, HV]"), gb_rows,
        _arg(state_pool, torch.float32, 0, "state_pool", "[slots, HV, V, K]"), slots,
        _arg(state_idx, torch.int32, n, "state_idx", "[num_seqs]"),
        _opt(cu_seqlens, torch.int32, n + 1, "cu_seqlens", "[num_seqs + 1]"), n, T,
        _arg(o, t16, T * HVV, "o", "[T, HV, V]"), _opt(intermediate, torch.float32, 0, "intermediate", "[chunks, HV, V, K]"),
        inter_chunks, *_space(workspace), _err(err_flag), _cur(stream))
    if st:
        _check(st, "kda_gdn_prefill")


def _gdn_rows(d, mixed_qkv, rows):
    shape, width = mixed_qkv.shape, 2 * d.H * d.K + d.HV * d.V
    if len(shape) != 2 or shape[0] < rows or shape[1] < width or mixed_qkv.stride(1) != 1:
        raise ValueError(f"mixed_qkv must be [>= {rows}, >= {width}] with unit column stride (got {tuple(shape)})")
    if mixed_qkv.dtype is not _t16(d) and mixed_qkv.dtype is not torch.int16:
        raise TypeError(f"mixed_qkv must be {_t16(d)} (got {mixed_qkv.dtype})")
    return _here(mixed_qkv)


def kda_gdn_decode_packed(d, gate: ScalarGate, mixed_qkv, a, b, state_pool, state_idx, o, err_flag=None,
                          stream=None):
    """One token per request, state in place; a, b [B, HV]."""
    B, t16 = mixed_qkv.shape[0], _t16(d)
    st = load().kda_gdn_decode_packed(
        d, gate.c(d), _gdn_rows(d, mixed_qkv, B), mixed_qkv.stride(0), _gate_rows(d, gate, a, B),
        _arg(b, t16, B * d.HV, "b", "[B, HV]"), B, _arg(state_pool, torch.float32, 0, "state_pool", "[slots, HV, V, K]"),
        _pool_slots(d, state_pool), _arg(state_idx, torch.int32, B, "state_idx", "[B]"),
        _arg(o, t16, B * d.HV * d.V, "o", "[B, HV, V]"), _err(err_flag), _cur(stream))
    if st:
        _check(st, "kda_gdn_decode_packed")


def _gdn_verify(name, call, d, gate, mixed_qkv, a, b, B, T, parents, state_pool, state_idx, o, snapshots, err_flag,
                stream):
    B, T = int(B), int(T)
    rows, t16 = B * T, _t16(d)
    st = call(
        d, gate.c(d), _gdn_rows(d, mixed_qkv, rows), mixed_qkv.stride(0), _gate_rows(d, gate, a, rows),
        _arg(b, t16, rows * d.HV, "b", "[B * T, HV]"), B, T, *parents,
        _arg(state_pool, torch.float32, 0, "state_pool", "[slots, HV, V, K]"), _pool_slots(d, state_pool),
        _arg(state_idx, torch.int32, B, "state_idx", "[B]"), _arg(o, t16, rows * d.HV * d.V, "o", "[B, T, HV, V]"),
        _arg(snapshots, torch.float32, rows * d.HV * d.V * d.K, "snapshots", "[B, T, HV, V, K]"), _err(err_flag),
        _cur(stream))
    if st:
        _check(st, name)


def kda_gdn_verify_chain(d, gate: ScalarGate, mixed_qkv, a, b, B, T, state_pool, state_idx, o, snapshots,
                         err_flag=None, stream=None):
    """Chain verify; snapshots as kda_verify_chain's, for kda_commit."""
    _gdn_verify("kda_gdn_verify_chain", load().kda_gdn_verify_chain, d, gate, mixed_qkv, a, b, B, T, (), state_pool,
                state_idx, o, snapshots, err_flag, stream)


def kda_gdn_verify_tree(d, gate: ScalarGate, mixed_qkv, a, b, B, T, parent_idx, state_pool, state_idx, o,
                        snapshots, err_flag=None, stream=None):
    """Tree verify; parent_idx [B, T] int32."""
    _gdn_verify("kda_gdn_verify_tree", load().kda_gdn_verify_tree, d, gate, mixed_qkv, a, b, B, T,
                (_arg(parent_idx, torch.int32, B * T, "parent_idx", "[B, T]"),), state_pool, state_idx, o, snapshots,
                err_flag, stream)


# -- verification of drafted tokens ------------------------------------------

_PROBS = {torch.float32: KDA_DTYPE_F32, torch.bfloat16: KDA_DTYPE_BF16, torch.float16: KDA_DTYPE_F16}


def _probs(t, dtype, name, B, T):
    """Pointer and row stride of probabilities [B, T, vocab]: the rows may be
    padded, but have one stride throughout."""
    shape, (s0, s1, s2) = t.shape, t.stride()
    V = shape[2]
    stride = s1 if T > 1 else s0 if B > 1 else V
    if shape[0] != B or shape[1] != T or (V > 1 and s2 != 1):
        raise ValueError(f"{name} must be [B, T, vocab] = [{B}, {T}, *] with dense rows (got {tuple(shape)})")
    if (B > 1 and s0 != T * stride) or stride < V:
        raise ValueError(f"the rows of {name} must lie one stride apart (got strides {(s0, s1, s2)})")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    return _here(t), stride


def _accept_sizes(target, tokens):
    if tokens.dim() != 2 or target.dim() != 3:
        raise ValueError(f"target must be [B, T, vocab] and tokens [B, T] (got {tuple(target.shape)}, "
                         f"{tuple(tokens.shape)})")
    if target.dtype not in _PROBS:
        raise TypeError(f"target must be float32, bfloat16 or float16 (got {target.dtype})")
    return tokens.shape[0], tokens.shape[1], target.shape[2]


def kda_accept_chain(target, draft, tokens, uniforms, accepted, next_token, lengths=None, err_flag=None,
                     stream=None):
    """Which drafted tokens stand, and the token behind them (see kda.h).
    target [B,T,vocab] and draft [B,T-1,vocab] (or None) probabilities of one
    element type, rows possibly padded; tokens [B,T] int32, uniforms [B,T] fp32,
    lengths [B] int32 or None; accepted [B] int32 (for kda_commit) and
    next_token [B] int32 (written)."""
    B, T, V = _accept_sizes(target, tokens)
    dtype, i32 = target.dtype, torch.int32
    p, p_stride = _probs(target, dtype, "target", B, T)
    q, q_stride = None, 0
    if draft is not None and T > 1:
        if draft.dim() != 3 or draft.shape[2] != V:
            raise ValueError("draft must have target's vocabulary")
        q, q_stride = _probs(draft, dtype, "draft", B, T - 1)
    st = load().kda_accept_chain(
        _PROBS[dtype], p, p_stride, q, q_stride, _arg(tokens, i32, B * T, "tokens", "[B, T]"),
        _arg(uniforms, torch.float32, B * T, "uniforms", "[B, T]"), _opt(lengths, i32, B, "lengths", "[B]"), B, T, V,
        _arg(accepted, i32, B, "accepted", "[B]"), _arg(next_token, i32, B, "next_token", "[B]"), _err(err_flag),
        _cur(stream))
    if st:
        _check(st, "kda_accept_chain")


def kda_accept_tree(target, tokens, parent_idx, uniforms, accepted, path, next_token, lengths=None, err_flag=None,
                    stream=None):
    """As kda_accept_chain for a tree proposed without probabilities:
    parent_idx [B,T] int32; path [B,T] int32 (written)."""
    B, T, V = _accept_sizes(target, tokens)
    dtype, i32 = target.dtype, torch.int32
    p, p_stride = _probs(target, dtype, "target", B, T)
    st = load().kda_accept_tree(
        _PROBS[dtype], p, p_stride, _arg(tokens, i32, B * T, "tokens", "[B, T]"),
        _arg(parent_idx, i32, B * T, "parent_idx", "[B, T]"), _arg(uniforms, torch.float32, B * T, "uniforms", "[B, T]"),
        _opt(lengths, i32, B, "lengths", "[B]"), B, T, V, _arg(accepted, i32, B, "accepted", "[B]"),
        _arg(path, i32, B * T, "path", "[B, T]"), _arg(next_token, i32, B, "next_token", "[B]"), _err(err_flag),
        _cur(stream))
    if st:
        _check(st, "kda_accept_tree")


# -- pages of a state pool ---------------------------------------------------


def _pages(pool):
    """Pages of a pool tensor [layers, slots, ...] whose slots are dense; the
    layers may lie further apart."""
    shape, size = pool.shape, pool.element_size()
    if len(shape) < 3:
        raise ValueError(f"pool must be [layers, slots, ...] (got {tuple(shape)})")
    base, page = _here(pool), 1
    for n in shape[2:]:
        page *= n
    if not pool.is_contiguous() and shape[0] > 0 and not pool[0].is_contiguous():
        raise ValueError("the slots of a layer must be dense")
    stride = pool.stride(0) if shape[0] > 1 else page * shape[1]
    return kda_pages(base, page * size, stride * size, shape[0], shape[1])


def _list(t, name):
    """Pointer of an int32 list."""
    if t.dim() != 1:
        raise ValueError(f"{name} must be a list [n] (got {tuple(t.shape)})")
    return _arg(t, torch.int32, 0, name, "[n]")


def _used(used, slots):
    return _arg(used, torch.bool if used.dtype is torch.bool else torch.uint8, slots, "used", "[slots]")


def kda_pool_copy(pool, src, dst, err_flag=None, stream=None):
    """pool[:, dst[i]] <- pool[:, src[i]]; pool [layers, slots, ...]."""
    n = src.shape[0]
    if dst.shape[0] != n:
        raise ValueError("src and dst must have one length")
    st = load().kda_pool_copy(_pages(pool), _list(src, "src"), _list(dst, "dst"), n, _err(err_flag), _cur(stream))
    if st:
        _check(st, "kda_pool_copy")


def kda_pool_free(used, table, rows, err_flag=None, stream=None):
    """Frees the pages of table rows `rows` and sets the rows to -1."""
    slots = used.shape[0]
    st = load().kda_pool_free(_used(used, slots), slots, _list(table, "table"), table.shape[0], _list(rows, "rows"),
                              rows.shape[0], _err(err_flag), _cur(stream))
    if st:
        _check(st, "kda_pool_free")


def kda_pool_compact(pool, used, table, count, err_flag=None, stream=None):
    """Moves the used pages to slots 0 .. count-1; table, used and count [1]
    int32 follow."""
    pages = _pages(pool)
    st = load().kda_pool_compact(pages, _used(used, pages.slots), _list(table, "table"), table.shape[0],
                                 _arg(count, torch.int32, 1, "count", "[1]"), _err(err_flag), _cur(stream))
    if st:
        _check(st, "kda_pool_compact")


def kda_pool_fork(pool, used, table, parents, rows, children=None, err_flag=None, stream=None):
    """Table row rows[i] gets the lowest free page, a copy of the page of row
    parents[i] (zeros where that is -1); returns children [n] int32, the slots
    given."""
    n = rows.shape[0]
    if parents.shape[0] != n:
        raise ValueError("parents and rows must have one length")
    if children is None:
        children = _new(n, torch.int32, rows.device, stream)
    pages = _pages(pool)
    st = load().kda_pool_fork(pages, _used(used, pages.slots), _list(table, "table"), table.shape[0],
                              _list(parents, "parents"), _list(rows, "rows"), n,
                              _arg(children, torch.int32, n, "children", "[n]"), _err(err_flag), _cur(stream))
    if st:
        _check(st, "kda_pool_fork")
    return children


# -- linear attention with one decay per value head ---------------------------


_F32, _I32 = torch.float32, torch.int32


def _lin_gate(gate, a, rows, HV, t16):
    """(kda_scalar_gate, gate input [>= rows, HV] or None where the heads' decay is fixed)."""
    A_log, bias = gate.A_log, gate.dt_bias
    g = kda_scalar_gate(None if A_log is None else _arg(A_log, _F32, HV, "A_log", "[HV]"),
                        None if bias is None else _arg(bias, _F32, HV, "dt_bias", "[HV]"), 0, 1 if gate.use_qk_l2norm else 0,
                        gate.scale)
    if a is None:
        return g, None
    if a.shape[-1] != HV:
        raise ValueError(f"`a` must have shape [rows, HV] = [{rows}, {HV}] (got {tuple(a.shape)})")
    return g, _arg(a, _F32 if A_log is None else t16, rows * HV, "a", "[rows, HV]")


def _lin_packed(d, gate, mixed_qkv, a, rows, B, state_pool, state_idx, o):
    """What the packed calls have in common, checked: the arguments up to the gate
    input, the pool and what goes with it, and a token's values."""
    load()
    H, HV, K, V, t16 = d.H, d.HV, d.K, d.V, _t16(d)
    qkv = _rows(mixed_qkv, t16, rows, 2 * H * K + HV * V) or (_gdn_rows(d, mixed_qkv, rows), mixed_qkv.stride(0))
    g, gate_rows = _lin_gate(gate, a, rows, HV, t16)
    return (d, g, *qkv, gate_rows), \
        (*_pool(d, state_pool, HV, V, K), _arg(state_idx, _I32, B, "state_idx", "[B]"),
         _arg(o, t16, rows * HV * V, "o", "[rows, HV, V]")), HV * V * K


def kda_lin_prefill_workspace_size(d: kda_dims, num_seqs: int, total_tokens: int) -> int:
    return int(load().kda_lin_prefill_workspace_size(d, int(num_seqs), int(total_tokens)))


def kda_lin_prefill(d, gate: ScalarGate, q, k, v, a, state_pool, state_idx, cu_seqlens, num_seqs, o, workspace=None,
                    err_flag=None, stream=None):
    """Varlen prefill (see kda.h).  q,k [T,H,K], v [T,HV,V], a [gate_rows,HV] or
    None (a head's decay is -exp(A_log) for every token); state_pool
    [slots,HV,V,K] fp32 (in place); o [T,HV,V] (written)."""
    lib, t16, HV, V = load(), _t16(d), d.HV, d.V
    T, n = q.shape[0], int(num_seqs)
    gate_rows = T if a is None else a.shape[0]
    HK, HVV = d.H * d.K, HV * V
    pool = _pool(d, state_pool, HV, V, d.K)
    g, rows = _lin_gate(gate, a, gate_rows, HV, t16)
    space = None, 0
    if workspace is None:
        need = lib.kda_lin_prefill_workspace_size(d, n, T)
        if need:
            workspace = _new(need, torch.uint8, q.device, stream)
            space = workspace.data_ptr(), need
    else:
        space = _space(workspace)
    st = lib.kda_lin_prefill(
        d, g, _arg(q, t16, T * HK, "q", "[T, H, K]"), _arg(k, t16, T * HK, "k", "[T, H, K]"),
        _arg(v, t16, T * HVV, "v", "[T, HV, V]"), rows, gate_rows,
        *pool, _arg(state_idx, _I32, n, "state_idx", "[num_seqs]"),
        None if cu_seqlens is None else _arg(cu_seqlens, _I32, n + 1, "cu_seqlens", "[num_seqs + 1]"), n, T,
        _arg(o, t16, T * HVV, "o", "[T, HV, V]"), *space, _err(err_flag), _cur(stream))
    if st:
        _check(st, "kda_lin_prefill")


def kda_lin_decode_packed(d, gate: ScalarGate, mixed_qkv, a, state_pool, state_idx, o, err_flag=None, stream=None):
    """One token per request, state in place; a [B, HV] or None."""
    B = mixed_qkv.shape[0]
    head, pool, _ = _lin_packed(d, gate, mixed_qkv, a, B, B, state_pool, state_idx, o)
    st = load().kda_lin_decode_packed(*head, B, *pool, _err(err_flag), _cur(stream))
    if st:
        _check(st, "kda_lin_decode_packed")


def _lin_verify(name, call, d, gate, mixed_qkv, a, B, T, parents, state_pool, state_idx, o, snapshots, err_flag, stream):
    rows = B * T
    head, pool, values = _lin_packed(d, gate, mixed_qkv, a, rows, B, state_pool, state_idx, o)
    st = call(*head, B, T, *parents, *pool, _arg(snapshots, _F32, rows * values, "snapshots", "[B, T, HV, V, K]"),
              _err(err_flag), _cur(stream))
    if st:
        _check(st, name)


def kda_lin_verify_chain(d, gate: ScalarGate, mixed_qkv, a, B, T, state_pool, state_idx, o, snapshots, err_flag=None,
                         stream=None):
    """Chain verify; snapshots as kda_verify_chain's, for kda_commit."""
    _lin_verify("kda_lin_verify_chain", load().kda_lin_verify_chain, d, gate, mixed_qkv, a, int(B), int(T), (), state_pool,
                state_idx, o, snapshots, err_flag, stream)


def kda_lin_verify_tree(d, gate: ScalarGate, mixed_qkv, a, B, T, parent_idx, state_pool, state_idx, o, snapshots,
                        err_flag=None, stream=None):
    """Tree verify; parent_idx [B, T] int32."""
    B, T = int(B), int(T)
    _lin_verify("kda_lin_verify_tree", load().kda_lin_verify_tree, d, gate, mixed_qkv, a, B, T,
                (_arg(parent_idx, _I32, B * T, "parent_idx", "[B, T]"),), state_pool, state_idx, o, snapshots, err_flag,
                stream)


# -- log probabilities of given tokens -----------------------------------------


def kda_token_logprobs(logits, tokens, logprobs, entropy=None, top_tokens=None, top_logprobs=None, err_flag=None,
                       stream=None):
    """Log probabilities of tokens [rows] int32 under logits [rows, vocab] (float32,
    bfloat16 or float16, rows possibly padded), see kda.h.  Written: logprobs
    [rows] fp32; entropy [rows] fp32, top_tokens [rows, top] int32 and
    top_logprobs [rows, top] fp32 where given."""
    shape, dtype = logits.shape, _PROBS.get(logits.dtype)
    if len(shape) != 2 or tokens.dim() != 1 or tokens.shape[0] != shape[0]:
        raise ValueError(f"logits must be [rows, vocab] and tokens [rows] (got {tuple(shape)}, {tuple(tokens.shape)})")
    if dtype is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16 (got {logits.dtype})")
    lib, (rows, V) = load(), shape
    at = _rows(logits, logits.dtype, rows, V)
    if at is None:  # (rows of one token may be apart)
        unit = logits.stride(1)
        if V > 1 and unit != 1:
            raise ValueError(f"the rows of logits must be dense (got strides {logits.stride()})")
        at = _here(logits), logits.stride(0)
    x, stride = at
    if rows <= 1:
        stride = V
    if stride < V:
        raise ValueError(f"the rows of logits must be dense (got strides {logits.stride()})")
    top, best, best_lp = 0, None, None
    if top_tokens is not None or top_logprobs is not None:
        if top_tokens is None or top_logprobs is None or top_tokens.dim() != 2 or top_tokens.shape != top_logprobs.shape or \
                top_tokens.shape[0] != rows:
            raise ValueError("top_tokens and top_logprobs must both be [rows, top]")
        top = top_tokens.shape[1]
        best = _arg(top_tokens, _I32, rows * top, "top_tokens", "[rows, top]")
        best_lp = _arg(top_logprobs, _F32, rows * top, "top_logprobs", "[rows, top]")
    st = lib.kda_token_logprobs(
        dtype, x, stride, _arg(tokens, _I32, rows, "tokens", "[rows]"), rows, V,
        _arg(logprobs, _F32, rows, "logprobs", "[rows]"),
        None if entropy is None else _arg(entropy, _F32, rows, "entropy", "[rows]"), top, best, best_lp, _err(err_flag),
        _cur(stream))
    if st:
        _check(st, "kda_token_logprobs")


# -- pages kept in 8 or 4 bits ---------------------------------------------------


def _archive(name, call, pool, codes, scales, src, dst, err_flag, stream):
    """A call on pages of a pool and the archive that keeps them: codes int8
    [slots, layers, .., K] (8 bits) or uint8 [slots, layers, .., K / 2] (4 bits,
    two codes a byte), scales fp32 with a scale for every 128 or 32 values."""
    kind, pairs, kept, held = codes.dtype, src.shape, codes.shape, scales.shape
    if pool.dtype is not _F32:
        raise TypeError(f"pool must be float32 (got {pool.dtype})")
    if kind is not torch.int8 and kind is not torch.uint8:
        raise TypeError(f"codes must be int8 (8 bits) or uint8 (4 bits) (got {kind})")
    if len(pairs) != 1 or dst.shape != pairs:
        raise ValueError(f"src and dst must be lists of one length (got {tuple(pairs)}, {tuple(dst.shape)})")
    pages = _pages(pool)
    bits, group = (8, 128) if kind is torch.int8 else (4, 32)
    slots = kept[0] if len(kept) else 0
    all_slots = pool.shape[1]
    values = pool.numel() // all_slots if all_slots else 0  # of a page, in all layers
    n = values * bits // 8
    if slots != (held[0] if len(held) else 0) or (all_slots and (codes.numel() != slots * n or scales.numel() * group != slots * values)):
        raise ValueError(f"codes and scales must hold {n} bytes and {values // group} scales a page "
                         f"(got {tuple(kept)}, {tuple(held)})")
    n = pairs[0]
    st = call(pages, kda_archive(_arg(codes, kind, 0, "codes", "[slots, layers, ..]"),
                                 _arg(scales, _F32, 0, "scales", "[slots, layers, ..]"), bits, slots),
              _arg(src, _I32, n, "src", "[n]"), _arg(dst, _I32, n, "dst", "[n]"), n, _err(err_flag), _cur(stream))
    if st:
        _check(st, name)


def kda_pool_store(pool, codes, scales, src, dst, err_flag=None, stream=None):
    """Archive page dst[i] <- pool[:, src[i]]; pool [layers, slots, ...] fp32, codes
    and scales as in _archive."""
    _archive("kda_pool_store", load().kda_pool_store, pool, codes, scales, src, dst, err_flag, stream)


def kda_pool_load(codes, scales, pool, src, dst, err_flag=None, stream=None):
    """pool[:, dst[i]] <- archive page src[i]."""
    _archive("kda_pool_load", load().kda_pool_load, pool, codes, scales, src, dst, err_flag, stream)
