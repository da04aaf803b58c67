// gdn_recurrent.cu -- the gated delta rule with one decay per value head,
// token by token: packed decode, chain and tree verify.
//
// Per value head, with S kept transposed in the pool ([V][K], K contiguous),
// raw keys and queries k, q and their inverse norms r_k, r_q:
//   p = S k, s = S q           (before the token)
//   c = r_k beta (v - e^g r_k p)
//   S <- e^g S + c k^T,  o = scale r_q (e^g s + c (k.q))
// Because the decay is one number, it and both norms stay outside the dot
// products: both products run on the state as it was loaded, side by side,
// and one reduction per token gives everything (p, s, k.k, q.q, k.q).  No
// token value passes through shared memory and the kernel has no barrier.
//
// Bound by HBM: decode reads and writes each 64 KiB head state once, verify
// reads it once and writes a snapshot per token.  A CTA of 4 warps owns
// 16 * GROUPS rows of S; a warp steps 4 rows at a time, 8 lanes per row, each
// lane holding 16 key channels as four float4, so that every 128-bit access
// of a warp covers four whole 128-byte segments.
// Measured (in a graph, on three sets of buffers in turn): decode of 48 requests,
// 32 heads, 31.9 us, 6.3 TB/s or 93% of a copy's rate; one request, 16 heads, 2.4
// us, a launch's latency; chain verify 16 x 6, 16 heads, 22 us, 5.4 TB/s or 80%
// (six of its seven parts are writes), tree 27.1 with random parents.
#include "kda_host.h"

namespace kda {
namespace {

enum GdnMode { kGdnDecode = 0, kGdnChain = 1, kGdnTree = 2 };

struct GdnStepArgs {
  ScalarGateArgs gate;
  int H, HV, G;  // G = HV / H
  const kda_bf16 *q, *k, *v;                // row 0 of each
  int64_t q_stride, k_stride, v_stride;     // elements between token rows
  const void* a;
  const kda_bf16* b;
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

// What one lane needs of a token: its 16 channels of q and k, the v of its
// rows, the gate input and beta of the head.
template <int GROUPS>
struct Token {
  uint2 q[4], k[4];
  uint16_t v[GROUPS];
  uint16_t b;
  ushort2 a;
  int parent;
};

template <int MODE, int GROUPS, bool F16>
__global__ void __launch_bounds__(128) gdn_recurrent_kernel(const GdnStepArgs args) {
  constexpr int K = kHeadDim, V = kHeadDim, kRowBlocks = V / (16 * GROUPS);
  const int rb = blockIdx.x % kRowBlocks;
  const int unit = blockIdx.x / kRowBlocks;
  const int r = unit / args.HV, h = unit % args.HV;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane & 7;
  const int row0 = rb * (16 * GROUPS) + warp * (4 * GROUPS) + (lane >> 3);
  const int HV = args.HV;
  const bool reporter = tid == 0 && rb == 0 && h == 0;

  const int64_t t0 = (int64_t)r * args.T;
  const int T = MODE == kGdnDecode ? 1 : args.T;

  auto load = [&](int t, Token<GROUPS>& x) {
    const int64_t row = t0 + t;
    const kda_bf16* q = args.q + row * args.q_stride + (h / args.G) * K + sub * 4;
    const kda_bf16* k = args.k + row * args.k_stride + (h / args.G) * K + sub * 4;
    const kda_bf16* v = args.v + row * args.v_stride + h * V;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x.k[i] = __ldg(reinterpret_cast<const uint2*>(k + i * 32));
      x.q[i] = __ldg(reinterpret_cast<const uint2*>(q + i * 32));
    }
#pragma unroll
    for (int gi = 0; gi < GROUPS; ++gi) x.v[gi] = __ldg(v + row0 + gi * 4);
    x.b = __ldg(args.b + row * HV + h);
    x.a = scalar_gate_load(args.gate, args.a, row * HV + h);
    if (MODE == kGdnTree) x.parent = __ldg(args.parent + row);
  };
  Token<GROUPS> next;
  load(0, next);
  const ScalarGateArgs& ga = args.gate;
  const float neg_rate = ga.A_log ? -expf(ga.A_log[h]) : 0.f;
  const float bias = ga.dt_bias ? ga.dt_bias[h] : 0.f;

  const int slot = args.state_idx[r];
  const bool ok = slot >= -1 && slot < args.pool_slots;
  if (!ok && reporter) set_error(args.err_flag, KDA_DEVERR_SLOT);
  bool live = ok && slot >= 0;
  uint32_t keep = 0;  // tree: bit i, a later node reloads node i's snapshot (nodes from 32 on: taken for granted)
  if (MODE == kGdnTree && live) {  // every warp checks the request's parents for itself
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
  // A chain's snapshots are not read again here (streamed: 4 x 6 tokens 7.0 instead
  // of 8.4 us); a tree's stay in L1 where a later node starts from them.
  auto store_state = [&](float* dst, bool again) {
#pragma unroll
    for (int gi = 0; gi < GROUPS; ++gi)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float4* at = reinterpret_cast<float4*>(dst + gi * 4 * K + i * 32);
        if (MODE == kGdnChain)
          __stcs(at, S[gi][i]);
        else if (MODE == kGdnDecode)
          *at = S[gi][i];
        else if (again)
          st_keep_l1(dst + gi * 4 * K + i * 32, S[gi][i]);
        else
          st_skip_l1(dst + gi * 4 * K + i * 32, S[gi][i]);
      }
  };
  load_state(root);

  for (int t = 0; t < T; ++t) {
    const Token<GROUPS> x = next;
    if (t + 1 < T) load(t + 1, next);
    const int64_t row = t0 + t;
    if (MODE == kGdnTree && t > 0) {
      const int p = x.parent;
      // the parent's snapshot was written by this same thread
      if (p != t - 1)
        load_state(p < 0 ? root : args.snapshots + (((size_t)t0 + p) * HV + h) * head_elems + (size_t)row0 * K + sub * 4);
    }
    float4 q[4], k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k[i] = in16x4_to_f4<F16>(x.k[i]);
      q[i] = in16x4_to_f4<F16>(x.q[i]);
    }
    float red[3 + 2 * GROUPS];
    red[0] = dot16(k, k);
    red[1] = dot16(q, q);
    red[2] = dot16(k, q);
#pragma unroll
    for (int gi = 0; gi < GROUPS; ++gi) {
      red[3 + 2 * gi] = dot16(S[gi], k);
      red[4 + 2 * gi] = dot16(S[gi], q);
    }
#pragma unroll
    for (int m = 1; m < 8; m <<= 1)
#pragma unroll
      for (int j = 0; j < 3 + 2 * GROUPS; ++j) red[j] += __shfl_xor_sync(0xffffffffu, red[j], m);
    const float alpha = expf(scalar_log_decay<F16>(ga, x.a, neg_rate, bias));
    const float bv = in16_to_float<F16>(x.b);
    const float beta = ga.beta_is_raw ? sigmoidf_(bv) : bv;
    const float rk = ga.use_qk_l2norm ? rsqrtf(red[0] + kNormEps) : 1.f;
    const float rq = ga.scale * (ga.use_qk_l2norm ? rsqrtf(red[1] + kNormEps) : 1.f);
#pragma unroll
    for (int gi = 0; gi < GROUPS; ++gi) {
      const float c = rk * beta * (in16_to_float<F16>(x.v[gi]) - alpha * rk * red[3 + 2 * gi]);
      const float2 c2 = make_float2(c, c), al2 = make_float2(alpha, alpha);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 lo = fma2(make_float2(k[i].x, k[i].y), c2, mul2(make_float2(S[gi][i].x, S[gi][i].y), al2));
        const float2 hi = fma2(make_float2(k[i].z, k[i].w), c2, mul2(make_float2(S[gi][i].z, S[gi][i].w), al2));
        S[gi][i] = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
      if (sub == 0)
        args.o[(row * HV + h) * V + row0 + gi * 4] = float_to_out16<F16>(rq * (alpha * red[4 + 2 * gi] + c * red[2]));
    }
    if (MODE == kGdnChain || MODE == kGdnTree)
      store_state(args.snapshots + ((size_t)row * HV + h) * head_elems + (size_t)row0 * K + sub * 4,
                  t >= 32 || (keep >> t & 1u));
  }
  if (MODE == kGdnDecode) store_state(root, false);
}

template <int MODE>
kda_status launch_gdn(const GdnStepArgs& a, int64_t requests, int dtype, cudaStream_t st) {
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
    (f16 ? gdn_recurrent_kernel<MODE, 1, true> : gdn_recurrent_kernel<MODE, 1, false>)<<<grid, 128, 0, st>>>(a);
  } else {
    const unsigned grid = (unsigned)(units * (kHeadDim / 32));
    (f16 ? gdn_recurrent_kernel<MODE, 2, true> : gdn_recurrent_kernel<MODE, 2, false>)<<<grid, 128, 0, st>>>(a);
  }
  const kda_status s = launch_status();
  record_stage(1, st);
  record_stage(2, st);
  return s;
}

kda_status check_gdn_packed(const kda_dims& d, const kda_scalar_gate& gate, const kda_bf16* mixed_qkv, int64_t row_stride,
                            const void* a, const kda_bf16* b, int B, const void* pool, int pool_slots,
                            const int32_t* state_idx, const kda_bf16* o, GdnStepArgs* out) {
  kda_status s = check_dims(d);
  if (s != KDA_OK) return s;
  if (!pool || !state_idx) return KDA_ERR_NULL_ARG;
  if (B < 0 || pool_slots < 0) return KDA_ERR_SHAPE;
  if (B > 0 && (!mixed_qkv || !a || !b || !o)) return KDA_ERR_NULL_ARG;
  if (row_stride < 2 * (int64_t)d.H * d.K + (int64_t)d.HV * d.V) return KDA_ERR_SHAPE;
  if (row_stride % 8 != 0 || !aligned16(mixed_qkv) || !aligned16(pool)) return KDA_ERR_ALIGNMENT;
  s = check_scalar_gate(gate, a, b, &out->gate);
  if (s != KDA_OK) return s;
  out->H = d.H;
  out->HV = d.HV;
  out->G = d.HV / d.H;
  out->q = mixed_qkv;
  out->k = mixed_qkv + (int64_t)d.H * d.K;
  out->v = mixed_qkv + 2 * (int64_t)d.H * d.K;
  out->q_stride = out->k_stride = out->v_stride = row_stride;
  out->a = a;
  out->b = b;
  out->pool_slots = pool_slots;
  out->state_idx = state_idx;
  return KDA_OK;
}

kda_status gdn_verify(kda_dims dims, kda_scalar_gate gate, const kda_bf16* mixed_qkv, int64_t row_stride, const void* a,
                      const kda_bf16* b, int B, int T, const int32_t* parent_idx, const float* state_pool, int pool_slots,
                      const int32_t* state_idx, kda_bf16* o, float* snapshots, int32_t* err_flag, void* stream, bool tree) {
  GdnStepArgs args{};
  kda_status s = check_gdn_packed(dims, gate, mixed_qkv, row_stride, a, b, B, state_pool, pool_slots, state_idx, o, &args);
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
  return tree ? launch_gdn<kGdnTree>(args, B, dims.dtype, st) : launch_gdn<kGdnChain>(args, B, dims.dtype, st);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_gdn_decode_packed(kda_dims dims, kda_scalar_gate gate, const kda_bf16* mixed_qkv,
                                            int64_t row_stride, const void* a, const kda_bf16* b, int B,
                                            float* state_pool, int pool_slots, const int32_t* state_idx, kda_bf16* o,
                                            int32_t* err_flag, void* stream) {
  GdnStepArgs args{};
  kda_status s = check_gdn_packed(dims, gate, mixed_qkv, row_stride, a, b, B, state_pool, pool_slots, state_idx, o, &args);
  if (s != KDA_OK) return s;
  if (B == 0) return KDA_OK;
  args.T = 1;
  args.pool = state_pool;
  args.o = o;
  args.err_flag = err_flag;
  return launch_gdn<kGdnDecode>(args, B, dims.dtype, static_cast<cudaStream_t>(stream));
}

extern "C" kda_status kda_gdn_verify_chain(kda_dims dims, kda_scalar_gate gate, const kda_bf16* mixed_qkv,
                                           int64_t row_stride, const void* a, const kda_bf16* b, int B, int T,
                                           const float* state_pool, int pool_slots, const int32_t* state_idx,
                                           kda_bf16* o, float* snapshots, int32_t* err_flag, void* stream) {
  return gdn_verify(dims, gate, mixed_qkv, row_stride, a, b, B, T, nullptr, state_pool, pool_slots, state_idx, o,
                    snapshots, err_flag, stream, false);
}

extern "C" kda_status kda_gdn_verify_tree(kda_dims dims, kda_scalar_gate gate, const kda_bf16* mixed_qkv,
                                          int64_t row_stride, const void* a, const kda_bf16* b, int B, int T,
                                          const int32_t* parent_idx, const float* state_pool, int pool_slots,
                                          const int32_t* state_idx, kda_bf16* o, float* snapshots, int32_t* err_flag,
                                          void* stream) {
  return gdn_verify(dims, gate, mixed_qkv, row_stride, a, b, B, T, parent_idx, state_pool, pool_slots, state_idx, o,
                    snapshots, err_flag, stream, true);
}
