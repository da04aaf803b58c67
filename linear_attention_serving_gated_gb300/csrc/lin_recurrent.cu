// lin_recurrent.cu -- linear attention with one decay per value head, token by
// token: packed decode, chain and tree verify.
//
// Per value head, with S kept transposed in the pool ([V][K], K contiguous),
// raw keys and queries k, q and their inverse norms r_k, r_q:
//   s = S q                    (before the token)
//   S <- e^g S + (r_k v) k^T,  o = scale r_q (e^g s + r_k (k.q) v)
// The decay is one number and norms only scale, so the product runs on the
// state as it was loaded and one reduction per token gives everything (s, k.k,
// q.q, k.q).  No token value passes through shared memory and the kernel has no
// barrier.
//
// Bound by HBM: decode reads and writes each 64 KiB head state once, verify
// reads it once and writes a snapshot per token.  A CTA of 4 warps owns
// 16 * GROUPS rows of S; a warp steps 4 rows at a time, 8 lanes per row, each
// lane holding 16 key channels as four float4, so that every 128-bit access
// of a warp covers four whole 128-byte segments.
//
// Decode of 48 requests at 32 value heads 31.9 us (6.3 TB/s), of one at 16 heads 2.3 us, a
// launch's time; chain verify of 16 x 6 at 16 heads 20.3 us (86% of a copy's rate, six
// of seven parts of it writes); tree verify of 4 x 10 at 8 heads 7.9 us, ten steps of
// 0.65 us one after the other in each of 256 CTAs, bound by the latency of a warp's
// instructions (16 lanes a row: 8.2; tokens or a parent's state loaded further ahead, no
// change).
#include "kda_host.h"
#include "lin.cuh"

namespace kda {
namespace {

enum LinMode { kLinDecode = 0, kLinChain = 1, kLinTree = 2 };

struct LinStepArgs {
  LinGateArgs gate;
  int H, HV, G;  // G = HV / H
  const kda_bf16 *q, *k, *v;             // row 0 of each
  int64_t q_stride, k_stride, v_stride;  // elements between token rows
  int T;
  const int32_t* parent;
  float* pool;
  int pool_slots;
  const int32_t* state_idx;
  kda_bf16* o;
  float* snapshots;
  int32_t* err_flag;
};

__device__ __forceinline__ float dot16(const float4 (&x)[4], const float4 (&y)[4]) {
  float2 a = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a = fma2(make_float2(x[i].x, x[i].y), make_float2(y[i].x, y[i].y), a);
    a = fma2(make_float2(x[i].z, x[i].w), make_float2(y[i].z, y[i].w), a);
  }
  return a.x + a.y;
}

// What one lane needs of a token: its 16 channels of q and k, the v of its rows
// and the head's gate input.
template <int GROUPS>
struct Token {
  uint2 q[4], k[4];
  uint16_t v[GROUPS];
  ushort2 a;
  int parent;
};

template <int MODE, int GROUPS, bool F16>
__global__ void __launch_bounds__(128) lin_recurrent_kernel(const LinStepArgs args) {
  constexpr int K = kHeadDim, V = kHeadDim, kRowBlocks = V / (16 * GROUPS);
  const int rb = blockIdx.x % kRowBlocks;
  const int unit = blockIdx.x / kRowBlocks;
  const int HV = args.HV;
  const int r = unit / HV, h = unit % HV;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane & 7;
  const int row0 = rb * (16 * GROUPS) + warp * (4 * GROUPS) + (lane >> 3);
  const bool reporter = tid == 0 && rb == 0 && h == 0;

  const int64_t t0 = (int64_t)r * args.T;
  const int T = MODE == kLinDecode ? 1 : args.T;

  // Tokens come one after the other: pointers that go on a row a step (with an index a
  // step's 64-bit products were a tenth of its instructions).  Decode has no next row, and
  // forms the address of its outputs late: with them held from the start it takes 72
  // registers instead of 76, 7 CTAs an SM instead of 6, and 35.5 us for 48 requests
  // instead of 31.5.
  const kda_bf16* kp = args.k + t0 * args.k_stride + (h / args.G) * K + sub * 4;
  const kda_bf16* qp = args.q + t0 * args.q_stride + (h / args.G) * K + sub * 4;
  const kda_bf16* vp = args.v + t0 * args.v_stride + h * V + row0;
  const int32_t* pp = args.parent + t0;
  int64_t gate_at = t0 * HV + h;
  auto load = [&](Token<GROUPS>& x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x.k[i] = __ldg(reinterpret_cast<const uint2*>(kp + i * 32));
      x.q[i] = __ldg(reinterpret_cast<const uint2*>(qp + i * 32));
    }
#pragma unroll
    for (int gi = 0; gi < GROUPS; ++gi) x.v[gi] = __ldg(vp + gi * 4);
    x.a = lin_gate_load(args.gate, gate_at);
    if (MODE == kLinTree) x.parent = __ldg(pp++);
    if (MODE != kLinDecode) {
      kp += args.k_stride, qp += args.q_stride, vp += args.v_stride;
      gate_at += HV;
    }
  };
  Token<GROUPS> next;
  load(next);
  const LinGateArgs& ga = args.gate;
  const float neg_rate = ga.A_log ? -expf(ga.A_log[h]) : 0.f;
  const float bias = ga.dt_bias ? ga.dt_bias[h] : 0.f;

  const int slot = args.state_idx[r];
  const bool ok = slot >= -1 && slot < args.pool_slots;
  if (!ok && reporter) set_error(args.err_flag, KDA_DEVERR_SLOT);
  bool live = ok && slot >= 0;
  uint32_t keep = 0;  // tree: bit i, a later node reloads node i's snapshot (nodes from 32 on: taken for granted)
  if (MODE == kLinTree && live) {  // every warp checks the request's parents for itself
    bool bad = false;
    for (int i = lane; i < T; i += 32) {
      const int p = args.parent[t0 + i];
      bad |= p < -1 || p >= i;
      if (p >= 0 && p < 32 && p != i - 1) keep |= 1u << p;
    }
    keep = __reduce_or_sync(0xffffffffu, keep);
    if (__any_sync(0xffffffffu, bad)) {
      if (reporter) set_error(args.err_flag, KDA_DEVERR_PARENT);
      live = false;
    }
  }
  if (!live) {  // padding or rejected: zero outputs, no state touched
    if (sub == 0)
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int gi = 0; gi < GROUPS; ++gi) args.o[((t0 + t) * HV + h) * V + row0 + gi * 4] = 0;
    return;
  }

  const size_t head_elems = (size_t)V * K;
  float* root = args.pool + ((size_t)slot * HV + h) * head_elems + (size_t)row0 * K + sub * 4;
  float4 S[GROUPS][4];
  auto load_state = [&](const float* src) {
#pragma unroll
    for (int gi = 0; gi < GROUPS; ++gi)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[gi][i] = *reinterpret_cast<const float4*>(src + gi * 4 * K + i * 32);
  };
  // A chain's snapshots are not read again here and are streamed; a tree's stay
  // in L1 where a later node starts from them.
  auto store_state = [&](float* dst, bool again) {
#pragma unroll
    for (int gi = 0; gi < GROUPS; ++gi)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* at = dst + gi * 4 * K + i * 32;
        if (MODE == kLinChain)
          __stcs(reinterpret_cast<float4*>(at), S[gi][i]);
        else if (MODE == kLinTree && again)
          st_keep_l1(at, S[gi][i]);
        else if (MODE == kLinTree)
          st_skip_l1(at, S[gi][i]);
        else
          *reinterpret_cast<float4*>(at) = S[gi][i];
      }
  };
  load_state(root);
  kda_bf16* o = args.o + (t0 * HV + h) * V + row0;
  float* snapshot = args.snapshots + ((size_t)t0 * HV + h) * head_elems + (size_t)row0 * K + sub * 4;

  constexpr int kUnroll = GROUPS == 1 && MODE != kLinDecode ? 2 : 1;
#pragma unroll kUnroll  // (two steps: 8.7 -> 7.9 us for the tree above)
  for (int t = 0; t < T; ++t) {
    const Token<GROUPS> x = next;
    if (t + 1 < T) load(next);
    if (MODE == kLinTree && t > 0) {
      const int p = x.parent;
      // the parent's snapshot was written by this same thread
      if (p != t - 1)
        load_state(p < 0 ? root : snapshot - (int64_t)(t - p) * (HV * (int64_t)head_elems));
    }
    float4 q[4], k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k[i] = in16x4_to_f4<F16>(x.k[i]);
      q[i] = in16x4_to_f4<F16>(x.q[i]);
    }
    float red[3 + GROUPS];
    red[0] = dot16(k, k);
    red[1] = dot16(q, q);
    red[2] = dot16(k, q);
#pragma unroll
    for (int gi = 0; gi < GROUPS; ++gi) red[3 + gi] = dot16(S[gi], q);
#pragma unroll
    for (int m = 1; m < 8; m <<= 1)
#pragma unroll
      for (int j = 0; j < 3 + GROUPS; ++j) red[j] += __shfl_xor_sync(0xffffffffu, red[j], m);
    const float alpha = expf(lin_log_decay<F16>(ga, x.a, neg_rate, bias));
    const float rk = ga.use_qk_l2norm ? rsqrtf(red[0] + kNormEps) : 1.f;
    const float rq = ga.scale * (ga.use_qk_l2norm ? rsqrtf(red[1] + kNormEps) : 1.f);
#pragma unroll
    for (int gi = 0; gi < GROUPS; ++gi) {
      const float c = rk * in16_to_float<F16>(x.v[gi]);
      const float2 c2 = make_float2(c, c), al2 = make_float2(alpha, alpha);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 lo = fma2(make_float2(k[i].x, k[i].y), c2, mul2(make_float2(S[gi][i].x, S[gi][i].y), al2));
        const float2 hi = fma2(make_float2(k[i].z, k[i].w), c2, mul2(make_float2(S[gi][i].z, S[gi][i].w), al2));
        S[gi][i] = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
      if (sub == 0)
        (MODE == kLinDecode ? args.o + (t0 * HV + h) * V + row0 : o)[gi * 4] = float_to_out16<F16>(rq * (alpha * red[3 + gi] + c * red[2]));
    }
    if (MODE == kLinChain || MODE == kLinTree)
      store_state(snapshot, t >= 32 || (keep >> t & 1u));
    o += HV * V;
    snapshot += HV * head_elems;
  }
  if (MODE == kLinDecode) store_state(root, false);
}

template <int MODE>
kda_status launch_lin(const LinStepArgs& a, int64_t requests, int dtype, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0) return KDA_ERR_CUDA;
  const int64_t units = requests * a.HV;
  if (units * (kHeadDim / 16) > INT32_MAX) return KDA_ERR_SHAPE;
  record_stage(0, st);
  const bool f16 = dtype == KDA_DTYPE_F16;
  // 16-row CTAs spread one request over 8 CTAs a head; past two CTAs a SM the
  // grid fills the SMs anyway and 32-row CTAs read each token half as often.
  if (units * (kHeadDim / 16) <= 2 * (int64_t)sms) {
    const unsigned grid = (unsigned)(units * (kHeadDim / 16));
    (f16 ? lin_recurrent_kernel<MODE, 1, true> : lin_recurrent_kernel<MODE, 1, false>)<<<grid, 128, 0, st>>>(a);
  } else {
    const unsigned grid = (unsigned)(units * (kHeadDim / 32));
    (f16 ? lin_recurrent_kernel<MODE, 2, true> : lin_recurrent_kernel<MODE, 2, false>)<<<grid, 128, 0, st>>>(a);
  }
  const kda_status s = launch_status();
  record_stage(1, st);
  record_stage(2, st);
  return s;
}

kda_status check_lin_packed(const kda_dims& d, const kda_scalar_gate& gate, const kda_bf16* mixed_qkv, int64_t row_stride,
                            const void* a, int B, const void* pool, int pool_slots, const int32_t* state_idx,
                            const kda_bf16* o, LinStepArgs* out) {
  kda_status s = check_dims(d);
  if (s != KDA_OK) return s;
  if (!pool || !state_idx) return KDA_ERR_NULL_ARG;
  if (B < 0 || pool_slots < 0) return KDA_ERR_SHAPE;
  if (B > 0 && (!mixed_qkv || !o)) return KDA_ERR_NULL_ARG;
  if (row_stride < 2 * (int64_t)d.H * d.K + (int64_t)d.HV * d.V) return KDA_ERR_SHAPE;
  if (row_stride % 8 != 0 || !aligned16(mixed_qkv) || !aligned16(pool)) return KDA_ERR_ALIGNMENT;
  s = check_lin_gate(gate, a, &out->gate);
  if (s != KDA_OK) return s;
  out->H = d.H;
  out->HV = d.HV;
  out->G = d.HV / d.H;
  out->q = mixed_qkv;
  out->k = mixed_qkv + (int64_t)d.H * d.K;
  out->v = mixed_qkv + 2 * (int64_t)d.H * d.K;
  out->q_stride = out->k_stride = out->v_stride = row_stride;
  out->pool_slots = pool_slots;
  out->state_idx = state_idx;
  return KDA_OK;
}

kda_status lin_verify(kda_dims dims, kda_scalar_gate gate, const kda_bf16* mixed_qkv, int64_t row_stride, const void* a,
                      int B, int T, const int32_t* parent_idx, const float* state_pool, int pool_slots,
                      const int32_t* state_idx, kda_bf16* o, float* snapshots, int32_t* err_flag, void* stream, bool tree) {
  LinStepArgs args{};
  kda_status s = check_lin_packed(dims, gate, mixed_qkv, row_stride, a, B, state_pool, pool_slots, state_idx, o, &args);
  if (s != KDA_OK) return s;
  if (T < 1) return KDA_ERR_SHAPE;
  if (B == 0) return KDA_OK;
  if (!snapshots || (tree && !parent_idx)) return KDA_ERR_NULL_ARG;
  if (!aligned16(snapshots)) return KDA_ERR_ALIGNMENT;
  args.T = T;
  args.parent = parent_idx;
  args.pool = const_cast<float*>(state_pool);  // read only in verify
  args.o = o;
  args.snapshots = snapshots;
  args.err_flag = err_flag;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return tree ? launch_lin<kLinTree>(args, B, dims.dtype, st) : launch_lin<kLinChain>(args, B, dims.dtype, st);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_lin_decode_packed(kda_dims dims, kda_scalar_gate gate, const kda_bf16* mixed_qkv,
                                            int64_t row_stride, const void* a, int B, float* state_pool, int pool_slots,
                                            const int32_t* state_idx, kda_bf16* o, int32_t* err_flag, void* stream) {
  LinStepArgs args{};
  kda_status s = check_lin_packed(dims, gate, mixed_qkv, row_stride, a, B, state_pool, pool_slots, state_idx, o, &args);
  if (s != KDA_OK) return s;
  if (B == 0) return KDA_OK;
  args.T = 1;
  args.pool = state_pool;
  args.o = o;
  args.err_flag = err_flag;
  return launch_lin<kLinDecode>(args, B, dims.dtype, static_cast<cudaStream_t>(stream));
}

extern "C" kda_status kda_lin_verify_chain(kda_dims dims, kda_scalar_gate gate, const kda_bf16* mixed_qkv,
                                           int64_t row_stride, const void* a, int B, int T, const float* state_pool,
                                           int pool_slots, const int32_t* state_idx, kda_bf16* o, float* snapshots,
                                           int32_t* err_flag, void* stream) {
  return lin_verify(dims, gate, mixed_qkv, row_stride, a, B, T, nullptr, state_pool, pool_slots, state_idx, o, snapshots,
                    err_flag, stream, false);
}

extern "C" kda_status kda_lin_verify_tree(kda_dims dims, kda_scalar_gate gate, const kda_bf16* mixed_qkv,
                                          int64_t row_stride, const void* a, int B, int T, const int32_t* parent_idx,
                                          const float* state_pool, int pool_slots, const int32_t* state_idx, kda_bf16* o,
                                          float* snapshots, int32_t* err_flag, void* stream) {
  return lin_verify(dims, gate, mixed_qkv, row_stride, a, B, T, parent_idx, state_pool, pool_slots, state_idx, o,
                    snapshots, err_flag, stream, true);
}
