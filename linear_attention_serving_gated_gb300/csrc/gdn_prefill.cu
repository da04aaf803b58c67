// gdn_prefill.cu -- chunked varlen prefill of the gated delta rule with one
// decay per value head, on tcgen05/TMEM.
//
// Per (sequence, value head), 64 tokens at a time.  c_i is the log-decay summed
// up to token i of the chunk, r_i the inverse norm of its key, S (K x V) the
// state before the chunk:
//   A_ij = beta_i r_i r_j e^(c_i - c_j) k_i.k_j  (j < i),   T = (I + A)^-1
//   X = K S,  Y_i = v_i - r_i e^(c_i) X_i,                  D = T Diag(beta) Y
//   O_i = scale rq_i e^(c_i) (Q S)_i + sum_(j <= i) P_ij D_j,
//         P_ij = scale rq_i r_j e^(c_i - c_j) q_i.k_j
//   S <- e^(c_last) S + sum_j e^(c_last - c_j) r_j k_j D_j^T
// One decay per head means that decays and norms only ever scale rows and
// columns of products, so the raw 16-bit q and k go into the tensor cores as
// they are: K K^T and Q K^T are exact up to FP32 sums, every exponent is of a
// difference c_i - c_j <= 0, and no decay is too strong for the chunk form.
//
// The state stays on the SM for the whole sequence and no workspace goes
// through memory.  A CTA owns DVS value columns of one head's state; three
// dependent products a chunk are its chain, and their latency, not bytes or
// flops, bounds a long sequence, so everything else is kept off it:
//   * 8 chain warps hold S in FP32 registers and turn each product's TMEM
//     accumulator into the next one's operand; products are
//       X  = [K; Q] S     128 x DVS x 128  (Q rows ride along for O)
//       D  = T Y          rows 0..63 of [T; P] x Y
//       dS = K^T D'       128 x DVS x 64, D'_j = e^(c_last - c_j) r_j D_j
//     then P D for the output while the state is being updated;
//   * prep groups of 4 warps, on alternating chunks, build T and P ahead of
//     the chain from [K; Q] K^T (tensor cores), with the 64 x 64 inverse by
//     blocks of 16 in FP32;
//   * one warp each issues the chain's products, [K; Q] K^T, and the TMA loads.
// Y, D' and S enter as MN-major operands: a thread writes one token's (or key
// channel's) columns with 16-byte stores, never a transpose.
//
// Precision: FP32 operands are split in two BF16 halves (hi + lo, 2^-16 left)
// wherever the state depends on them: S, T, Y and D'.  K and Q are BF16 already;
// FP16 ones are split exactly.  P alone is rounded to BF16 once (2^-9): it
// only enters the output, itself rounded to 16 bits.
#include <atomic>

#include "kda_host.h"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kC = 64;  // tokens per chunk
constexpr int kChainWarps = 8;
constexpr int kLdA = 68, kLdZ = 36;  // FP32 row strides: 16-byte aligned, rows on different banks

struct GdnPrefillArgs {
  ScalarGateArgs gate;
  int H, HV, G;
  const kda_bf16* v;
  const void* a;
  const kda_bf16* beta;
  float* pool;
  int pool_slots;
  const int32_t* state_idx;
  const int32_t* cu_seqlens;
  int num_seqs;
  int64_t total_tokens;
  kda_bf16* o;
  float* intermediate;
  int64_t inter_chunks;
  int32_t* err_flag;
};

struct GdnMaps {
  CUtensorMap q, k;
};

// Per prep group: what the chain warps read of a chunk (a, s, o, last) and what
// the group keeps for itself.
struct ChunkScalars {
  float a[kC];     // r_i e^(c_i)
  float s[kC];     // r_j e^(c_last - c_j), 0 past the sequence's end
  float o[kC];     // scale rq_i e^(c_i)
  float hi[kC], lo[kC];  // c_i = hi + lo
  float beta[kC], rk[kC];
  float last;      // e^(c_last)
  float pad[3];
};

template <int DVS, bool F16>
struct Cfg {
  static constexpr int kStages = DVS == 64 || F16 ? 2 : 3;  // chunks of K and Q in shared memory
  static constexpr int kGroups = F16 ? 1 : 2;               // prep groups
  static constexpr int kTiles = DVS * 2 / 64;  // 64-wide operand tiles: [hi], [lo], or one [hi | lo]
  static constexpr int kStageBytes = 32768 * (F16 ? 2 : 1);
  static constexpr int kS = kStages * kStageBytes;
  static constexpr int kTP = kS + kTiles * 16384;
  static constexpr int kTPBytes = 16384 + 8192;  // [T; P] hi, T lo
  static constexpr int kY = kTP + kGroups * kTPBytes;
  static constexpr int kD = kY + kTiles * 8192;
  static constexpr int kScratch = kD + kTiles * 8192;
  static constexpr int kScratchBytes = (kC * kLdA + 32 * kLdZ) * 4;
  static constexpr int kScalars = kScratch + kGroups * kScratchBytes;
  static constexpr int kEnd = kScalars + kGroups * (int)sizeof(ChunkScalars);
  static constexpr int kSmem = kEnd + 1024;  // alignment slack
  static constexpr int kPrepWarp = kChainWarps;
  static constexpr int kMmaWarp = kPrepWarp + 4 * kGroups;
  static constexpr int kThreads = (kMmaWarp + 3) * 32;
};

// TMEM columns
constexpr int kTmX = 0, kTmD = 64, kTmU = 128, kTmO = 192, kTmA = 320, kTmCols = 512;

struct Bars {
  uint64_t full[3], ready[3], free_[3];  // K/Q stage: landed, tail zeroed (or split), consumed
  uint64_t a_full[2];                    // [K; Q] K^T done
  uint64_t tp_ready[2], tp_free[2];      // T, P and the chunk's scalars
  uint64_t s_ready, x_full, y_ready, d_full, u_ready, v_ready, u_full;
  uint64_t o_full[2];
};

__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity));
}

// A warp's writes to shared memory are for the tensor core, and its TMEM reads
// are done: one arrival per warp.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  tc::fence_async_smem();
  tc::tc_fence_before();
  __syncwarp();
  if (lane == 0) arrive(bar);
}

// Barrier of a prep group's 128 threads that also tells whether any of them failed.
__device__ __forceinline__ bool group_any(int id, bool bad) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)bad), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }

// Eight FP32 values as BF16 hi and lo halves.
__device__ __forceinline__ void split8(const float* x, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * p], x[2 * p + 1]);
    h[p] = *reinterpret_cast<const uint32_t*>(&b);
    const __nv_bfloat162 c = __floats2bfloat162_rn(x[2 * p] - __uint_as_float(h[p] << 16),
                                                   x[2 * p + 1] - __uint_as_float(h[p] & 0xffff0000u));
    l[p] = *reinterpret_cast<const uint32_t*>(&c);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

__device__ __forceinline__ uint4 round8(const float* x) {
  uint32_t h[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * p], x[2 * p + 1]);
    h[p] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// 16-byte piece `piece` of 128-byte line `row` of a 128-byte-swizzled tile.
__device__ __forceinline__ uint4* line16(uint8_t* tile, int row, int piece) {
  return reinterpret_cast<uint4*>(tile + row * 128 + ((piece ^ (row & 7)) << 4));
}

// A row's values as operand halves: columns [half * N, half * N + N) of the CTA's
// DVS = 2 N, N = 32 in tiles [hi], [lo], N = 16 in one tile [hi | lo].
template <int N>
__device__ __forceinline__ void put_split(uint8_t* tiles, int tile_bytes, int row, int half, const float (&x)[N]) {
#pragma unroll
  for (int j = 0; j < N / 8; ++j) {
    uint4 hi, lo;
    split8(x + 8 * j, hi, lo);
    const int piece = half * (N / 8) + j;
    *line16(tiles, row, piece) = hi;
    if (N == 32)
      *line16(tiles + tile_bytes, row, piece) = lo;
    else
      *line16(tiles, row, 4 + piece) = lo;
  }
}

// A warp's accumulator columns of its half: 32 columns, or 16 of the hi product
// plus the same 16 of the lo product.
template <int N>
__device__ __forceinline__ void get_acc(uint32_t taddr, int half, float (&x)[N]) {
  uint32_t a[16], b[16];
  tc::tmem_ld16_async(taddr + half * N, a);
  tc::tmem_ld16_async(taddr + half * N + (N == 32 ? 16 : 32), b);
  tc::tmem_wait_ld();
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (N == 32) {
      x[j] = __uint_as_float(a[j]);
      x[(16 + j) % N] = __uint_as_float(b[j]);
    } else {
      x[j] = __uint_as_float(a[j]) + __uint_as_float(b[j]);
    }
  }
}

__device__ __forceinline__ int64_t seq_start(const GdnPrefillArgs& a, int n) {
  return a.cu_seqlens ? (int64_t)a.cu_seqlens[n] : a.total_tokens / a.num_seqs * n;
}

// (I + A)^-1 in place in `m` ([64][kLdA], A strictly lower, rest ignored above
// the diagonal blocks), 128 threads; z: [32][kLdZ] scratch.  Diagonal blocks of
// 16 by forward substitution, one warp each, a column per lane; then
// T21 = -T22 (A21 T11) for blocks of 16 and of 32.
__device__ __forceinline__ void invert64(float* m, float* z, int t, int bar_id) {
  const int warp = t >> 5, lane = t & 31;
  {
    float* d = m + warp * 16 * (kLdA + 1);
    const int col = lane & 15;
    float x[16];
    float4 row[4];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
      for (int j = 0; j < (i + 3) / 4; ++j) row[j] = *reinterpret_cast<const float4*>(d + i * kLdA + 4 * j);
      const float* r = reinterpret_cast<const float*>(row);
      float s0 = col == i ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) {
        if (j & 1) s1 = fmaf(-r[j], x[j], s1); else s0 = fmaf(-r[j], x[j], s0);
      }
      x[i] = s0 + s1;
    }
    __syncwarp();
    if (lane < 16)
#pragma unroll
      for (int i = 0; i < 16; ++i) d[i * kLdA + col] = x[i];
  }
  group_sync(bar_id);
  {  // blocks (1,0) and (3,2): 64 threads each, a row and 4 columns a thread
    const int p = t >> 6, r = (t & 63) >> 2, c = (t & 3) * 4;
    float* a21 = m + (32 * p + 16) * kLdA + 32 * p;
    const float* t11 = m + 32 * p * (kLdA + 1);
    const float* t22 = m + (32 * p + 16) * (kLdA + 1);
    float* zz = z + p * 16 * kLdZ;
    auto mul = [&](const float* left, const float* right, int ld) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k4 = 0; k4 < 4; ++k4) {
        const float4 l = *reinterpret_cast<const float4*>(left + 4 * k4);
        const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 b = *reinterpret_cast<const float4*>(right + (4 * k4 + e) * ld + c);
          acc.x = fmaf(lv[e], b.x, acc.x);
          acc.y = fmaf(lv[e], b.y, acc.y);
          acc.z = fmaf(lv[e], b.z, acc.z);
          acc.w = fmaf(lv[e], b.w, acc.w);
        }
      }
      return acc;
    };
    const float4 y = mul(a21 + r * kLdA, t11, kLdA);
    *reinterpret_cast<float4*>(zz + r * kLdZ + c) = y;
    group_sync(bar_id);
    const float4 w = mul(t22 + r * kLdA, zz, kLdZ);
    *reinterpret_cast<float4*>(a21 + r * kLdA + c) = make_float4(-w.x, -w.y, -w.z, -w.w);
  }
  group_sync(bar_id);
  {  // block (2..3, 0..1): 2 rows and 4 columns a thread
    const int r = (t >> 3) * 2, c = (t & 7) * 4;
    float* a21 = m + 32 * kLdA;
    auto mul = [&](const float* left, const float* right, int ld, float4 (&acc)[2]) {
      acc[0] = acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k4 = 0; k4 < 8; ++k4) {
        const float4 l0 = *reinterpret_cast<const float4*>(left + 4 * k4);
        const float4 l1 = *reinterpret_cast<const float4*>(left + kLdA + 4 * k4);
        const float v0[4] = {l0.x, l0.y, l0.z, l0.w}, v1[4] = {l1.x, l1.y, l1.z, l1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 b = *reinterpret_cast<const float4*>(right + (4 * k4 + e) * ld + c);
          acc[0].x = fmaf(v0[e], b.x, acc[0].x);
          acc[0].y = fmaf(v0[e], b.y, acc[0].y);
          acc[0].z = fmaf(v0[e], b.z, acc[0].z);
          acc[0].w = fmaf(v0[e], b.w, acc[0].w);
          acc[1].x = fmaf(v1[e], b.x, acc[1].x);
          acc[1].y = fmaf(v1[e], b.y, acc[1].y);
          acc[1].z = fmaf(v1[e], b.z, acc[1].z);
          acc[1].w = fmaf(v1[e], b.w, acc[1].w);
        }
      }
    };
    float4 acc[2];
    mul(a21 + r * kLdA, m, kLdA, acc);
    *reinterpret_cast<float4*>(z + r * kLdZ + c) = acc[0];
    *reinterpret_cast<float4*>(z + (r + 1) * kLdZ + c) = acc[1];
    group_sync(bar_id);
    mul(m + (32 + r) * kLdA + 32, z, kLdZ, acc);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      *reinterpret_cast<float4*>(a21 + (r + e) * kLdA + c) = make_float4(-acc[e].x, -acc[e].y, -acc[e].z, -acc[e].w);
  }
  group_sync(bar_id);
}

template <int DVS, bool F16>
__global__ void __launch_bounds__(Cfg<DVS, F16>::kThreads, 1)
    gdn_prefill_kernel(const GdnPrefillArgs args, const __grid_constant__ GdnMaps maps) {
  using C = Cfg<DVS, F16>;
  constexpr int N = DVS / 2;  // value columns per chain thread
  constexpr int kSlices = kHeadDim / DVS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int timed_out;
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slice = blockIdx.x % kSlices;
  const int unit = blockIdx.x / kSlices;
  const int h = unit % args.HV, n = unit / args.HV;
  const bool reporter = tid == 0 && slice == 0 && h == 0;

  const int64_t t0 = seq_start(args, n), t1 = seq_start(args, n + 1);
  if (t0 < 0 || t1 < t0 || t1 > args.total_tokens || (n == 0 && t0 != 0) ||
      (n == args.num_seqs - 1 && t1 != args.total_tokens)) {
    if (reporter) set_error(args.err_flag, KDA_DEVERR_SEQLENS);
    return;
  }
  const int L = (int)(t1 - t0);
  if (L == 0) return;
  const int slot = args.state_idx[n];
  if (slot < 0 || slot >= args.pool_slots) {  // padding or out of range: zero outputs, no state touched
    if (slot != -1 && reporter) set_error(args.err_flag, KDA_DEVERR_SLOT);
    constexpr int kPieces = DVS / 8;
    for (int64_t i = tid; i < (int64_t)L * kPieces; i += C::kThreads)
      *reinterpret_cast<uint4*>(args.o + ((t0 + i / kPieces) * args.HV + h) * kHeadDim + slice * DVS +
                                (i % kPieces) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int nch = (L + kC - 1) / kC;

  if (warp == C::kMmaWarp) tc::tmem_alloc(&tmem_slot, kTmCols);
  if (tid == 0) {
    timed_out = 0;
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(&bars.full[i], 1);
      tc::mbar_init(&bars.ready[i], 4);
      tc::mbar_init(&bars.free_[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.a_full[i], 1);
      tc::mbar_init(&bars.tp_ready[i], 4);
      tc::mbar_init(&bars.tp_free[i], 1 + kChainWarps);
      tc::mbar_init(&bars.o_full[i], 1);
    }
    tc::mbar_init(&bars.s_ready, kChainWarps);
    tc::mbar_init(&bars.x_full, 1);
    tc::mbar_init(&bars.y_ready, kChainWarps / 2);
    tc::mbar_init(&bars.d_full, 1);
    tc::mbar_init(&bars.u_ready, kChainWarps / 2);
    tc::mbar_init(&bars.v_ready, kChainWarps / 2);
    tc::mbar_init(&bars.u_full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  bool ok = true;

  if (warp < kChainWarps) {
    // ---------------------------------------------------------------- chain
    const int quad = warp & 3, half = warp >> 2;
    const bool krow = quad < 2;
    const int row = 32 * (quad & 1) + lane;    // token of the chunk (K rows, or Q rows)
    const int dk = 32 * quad + lane;           // key channel of the state
    const int col0 = slice * DVS + half * N;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    float* root = args.pool + (((size_t)slot * args.HV + h) * kHeadDim + col0) * kHeadDim + dk;
    float S[N];
#pragma unroll
    for (int j = 0; j < N; ++j) S[j] = root[j * kHeadDim];
    put_split<N>(smem + C::kS, 16384, dk, half, S);
    warp_arrive(&bars.s_ready, lane);
    int64_t cid = 0;  // record of this sequence's first chunk
    if (args.intermediate) {
      for (int m = lane; m < n; m += 32) {
        const int64_t len = seq_start(args, m + 1) - seq_start(args, m);
        cid += len > 0 ? (len + kC - 1) / kC : 0;
      }
#pragma unroll
      for (int m = 16; m; m >>= 1) cid += __shfl_xor_sync(0xffffffffu, cid, m);
    }
    auto load_v = [&](int c, uint4 (&v)[N / 8]) {
      const int t = c * kC + row;
#pragma unroll
      for (int j = 0; j < N / 8; ++j) v[j] = make_uint4(0, 0, 0, 0);
      if (krow && t < L) {
        const uint4* src = reinterpret_cast<const uint4*>(args.v + ((t0 + t) * args.HV + h) * kHeadDim + col0);
#pragma unroll
        for (int j = 0; j < N / 8; ++j) v[j] = __ldg(src + j);
      }
    };
    uint4 vraw[N / 8];
    load_v(0, vraw);
    for (int c = 0; c < nch && ok; ++c) {
      const int g = c % C::kGroups;
      const uint32_t gp = (uint32_t)(c / C::kGroups) & 1u, cp = (uint32_t)c & 1u;
      if (args.intermediate) {
        if (cid + c < args.inter_chunks) {
          float* dst = args.intermediate + (((size_t)(cid + c) * args.HV + h) * kHeadDim + col0) * kHeadDim + dk;
#pragma unroll
          for (int j = 0; j < N; ++j) dst[j * kHeadDim] = S[j];
        } else if (reporter) {
          set_error(args.err_flag, KDA_DEVERR_INTERMEDIATE);
        }
      }
      const ChunkScalars& sc = *reinterpret_cast<const ChunkScalars*>(smem + C::kScalars + g * sizeof(ChunkScalars));
      if (!(ok = warp_wait(&bars.tp_ready[g], gp))) break;
      const float last = sc.last, fa = krow ? sc.a[row] : sc.o[row], fs = sc.s[row];
      __syncwarp();
      if (lane == 0) arrive(&bars.tp_free[g]);
      if (!(ok = warp_wait(&bars.x_full, cp))) break;
      tc::tc_fence_after();
      float x[N];
      get_acc<N>(lanes + kTmX, half, x);
      if (krow) {
        // Y = v - r e^c (K S)
        const uint32_t* vw = reinterpret_cast<const uint32_t*>(vraw);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t w = vw[j / 2];
          float v;
          if constexpr (F16)
            v = in16_to_float<true>((uint16_t)(j & 1 ? w >> 16 : w & 0xffffu));
          else
            v = __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
          x[j] = fmaf(-fa, x[j], v);
        }
        put_split<N>(smem + C::kY, 8192, row, half, x);
        warp_arrive(&bars.y_ready, lane);
        if (c + 1 < nch) load_v(c + 1, vraw);
        if (!(ok = warp_wait(&bars.d_full, cp))) break;
        tc::tc_fence_after();
        get_acc<N>(lanes + kTmD, half, x);
        float y[N];
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = fs * x[j];
        put_split<N>(smem + C::kY, 8192, row, half, y);
        warp_arrive(&bars.u_ready, lane);
        put_split<N>(smem + C::kD, 8192, row, half, x);
        warp_arrive(&bars.v_ready, lane);
      }
      if (!(ok = warp_wait(&bars.u_full, cp))) break;
      tc::tc_fence_after();
      float u[N];
      get_acc<N>(lanes + kTmU, half, u);
#pragma unroll
      for (int j = 0; j < N; ++j) S[j] = fmaf(last, S[j], u[j]);
      if (c + 1 < nch) put_split<N>(smem + C::kS, 16384, dk, half, S);
      warp_arrive(&bars.s_ready, lane);
      if (!krow) {
        if (!(ok = warp_wait(&bars.o_full[c & 1], (uint32_t)(c >> 1) & 1u))) break;
        tc::tc_fence_after();
        get_acc<N>(lanes + kTmO + 64 * (c & 1), half, u);
        const int t = c * kC + row;
        if (t < L) {
          uint4* dst = reinterpret_cast<uint4*>(args.o + ((t0 + t) * args.HV + h) * kHeadDim + col0);
#pragma unroll
          for (int j = 0; j < N / 8; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_out16x2<F16>(fmaf(fa, x[8 * j + 2 * e], u[8 * j + 2 * e]),
                                       fmaf(fa, x[8 * j + 2 * e + 1], u[8 * j + 2 * e + 1]));
            dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
    if (ok)
#pragma unroll
      for (int j = 0; j < N; ++j) root[j * kHeadDim] = S[j];
  } else if (warp < C::kMmaWarp) {
    // ----------------------------------------------------------------- prep
    const int g = (warp - C::kPrepWarp) >> 2;
    const int t = tid - (C::kPrepWarp + 4 * g) * 32, quad = warp & 3;
    const int bar_id = 1 + g;
    const bool krow = quad < 2;
    const int i = 32 * (quad & 1) + lane;  // token of the chunk
    const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16) + kTmA + 64 * g;
    uint8_t* tp_hi = smem + C::kTP + g * C::kTPBytes;
    uint8_t* tp_lo = tp_hi + 16384;
    float* am = reinterpret_cast<float*>(smem + C::kScratch + g * C::kScratchBytes);
    float* zm = am + kC * kLdA;
    ChunkScalars& sc = *reinterpret_cast<ChunkScalars*>(smem + C::kScalars + g * sizeof(ChunkScalars));
    const ScalarGateArgs& ga = args.gate;
    const float neg_rate = ga.A_log ? -expf(ga.A_log[h]) : 0.f;
    const float bias = ga.dt_bias ? ga.dt_bias[h] : 0.f;
    // the gate warp's lane takes tokens 2 lane and 2 lane + 1
    float gl[2] = {0.f, 0.f}, be[2] = {0.f, 0.f};
    auto load_gate = [&](int c) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = c * kC + 2 * lane + e;
        gl[e] = be[e] = 0.f;
        if (c < nch && tok < L) {
          const int64_t at = (t0 + tok) * args.HV + h;
          gl[e] = scalar_log_decay<F16>(ga, args.a, at, neg_rate, bias);
          const float b = in16_to_float<F16>(args.beta[at]);
          be[e] = ga.beta_is_raw ? sigmoidf_(b) : b;
        }
      }
    };
    if (quad == 3) load_gate(g);
    for (int c = g; c < nch; c += C::kGroups) {
      const int k = c / C::kGroups, st = c % C::kStages;
      const int len = L - c * kC < kC ? L - c * kC : kC;
      uint8_t* kq = smem + st * C::kStageBytes;
      bool bad = !warp_wait(&bars.full[st], (uint32_t)(c / C::kStages) & 1u);
      const int row = krow ? i : 64 + i;  // row of [K; Q]
      float ss = 0.f;
      if constexpr (F16) {
        // FP16 rows as two BF16 halves (exact: 11 bits into 8 + 8), K rows past the end zero
        const bool drop = krow && i >= len;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            uint4* src = line16(kq + a * 16384, row, p);
            const uint4 w = *src;
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              f[e] = drop ? 0.f : in16_to_float<true>((uint16_t)(e & 1 ? ww[e / 2] >> 16 : ww[e / 2] & 0xffffu));
              ss = fmaf(f[e], f[e], ss);
            }
            uint4 hi, lo;
            split8(f, hi, lo);
            *src = hi;
            *line16(kq + 32768 + a * 16384, row, p) = lo;
          }
        }
      } else if (len < kC) {  // rows of the next sequence, or past the last: K rows zero
        for (int x = t; x < (kC - len) * 16; x += 128)
          *line16(kq + (x & 1) * 16384, len + x / 16, (x >> 1) & 7) = make_uint4(0, 0, 0, 0);
      }
      warp_arrive(&bars.ready[st], lane);
      if constexpr (!F16) {
        if (len < kC) group_sync(bar_id);  // other threads' zeros are read below
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const uint4 w = *line16(kq + a * 16384, row, p);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float f0 = __uint_as_float(ww[e] << 16), f1 = __uint_as_float(ww[e] & 0xffff0000u);
              ss = fmaf(f0, f0, fmaf(f1, f1, ss));
            }
          }
      }
      const float r = (krow ? 1.f : ga.scale) * (ga.use_qk_l2norm ? rsqrtf(ss + kNormEps) : 1.f);
      if (krow) sc.rk[i] = r;
      if (quad == 3) {  // running sums of the log-decays, in FP64, kept as two floats
        const double g0 = gl[0], g1 = g0 + (double)gl[1];
        double run = g1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const double up = __shfl_up_sync(0xffffffffu, run, d);
          if (lane >= d) run += up;
        }
        const double c1 = run, c0 = run - (double)gl[1];
        sc.hi[2 * lane] = (float)c0;
        sc.lo[2 * lane] = (float)(c0 - (double)(float)c0);
        sc.hi[2 * lane + 1] = (float)c1;
        sc.lo[2 * lane + 1] = (float)(c1 - (double)(float)c1);
        sc.beta[2 * lane] = be[0];
        sc.beta[2 * lane + 1] = be[1];
        load_gate(c + C::kGroups);
      }
      // the previous chunk's T, P and scalars of this group have been used
      if (k > 0) bad |= !warp_wait(&bars.tp_free[g], (uint32_t)(k - 1) & 1u);
      bad |= !warp_wait(&bars.a_full[g], (uint32_t)k & 1u);
      if (group_any(bar_id, bad)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const float ci_hi = sc.hi[i], ci_lo = sc.lo[i];
      const float ei = __expf(ci_hi + ci_lo);
      if (krow) {
        sc.a[i] = r * ei;
        sc.s[i] = i < len ? r * __expf((sc.hi[63] - ci_hi) + (sc.lo[63] - ci_lo)) : 0.f;
        if (i == 63) sc.last = ei;
      } else {
        sc.o[i] = r * ei;
      }
      const float ri = krow ? r * sc.beta[i] : r;
      const int top = 32 * (quad & 1) + 31;  // last row of this warp
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        float d[16];
        const bool any = 16 * jb <= top;
        if (any) {
          tc::tmem_ld16(acc + 16 * jb, d);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int j = 16 * jb + e;
            const float f = ri * sc.rk[j] * __expf((ci_hi - sc.hi[j]) + (ci_lo - sc.lo[j]));
            d[e] = (krow ? j < i : j <= i) ? f * d[e] : 0.f;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) d[e] = 0.f;
        }
        if (krow) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<float4*>(am + i * kLdA + 16 * jb + 4 * e) =
                make_float4(d[4 * e], d[4 * e + 1], d[4 * e + 2], d[4 * e + 3]);
        } else {
          *line16(tp_hi, 64 + i, 2 * jb) = round8(d);
          *line16(tp_hi, 64 + i, 2 * jb + 1) = round8(d + 8);
        }
      }
      tc::tc_fence_before();
      group_sync(bar_id);
      invert64(am, zm, t, bar_id);
      {  // T Diag(beta), half a row a thread
        const int ti = t >> 1, j0 = (t & 1) * 32;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int j = j0 + 8 * p + e;
            f[e] = j <= ti ? am[ti * kLdA + j] * sc.beta[j] : 0.f;
          }
          uint4 hi, lo;
          split8(f, hi, lo);
          *line16(tp_hi, ti, (j0 >> 3) + p) = hi;
          *line16(tp_lo, ti, (j0 >> 3) + p) = lo;
        }
      }
      warp_arrive(&bars.tp_ready[g], lane);
      group_sync(bar_id);  // the scratch and scalars are rewritten by the next chunk
    }
  } else if (warp == C::kMmaWarp) {
    // ----------------------------------------------------- the chain's products
    if (lane == 0) {
      constexpr uint32_t kIdX = tc::idesc_bf16_f32(128, 64) | tc::kIdescMnB;
      constexpr uint32_t kIdU = kIdX | tc::kIdescMnA;
      const uint32_t s_op = tc::smem_u32(smem + C::kS), y_op = tc::smem_u32(smem + C::kY),
                     d_op = tc::smem_u32(smem + C::kD);
      for (int c = 0; c < nch; ++c) {
        const int g = c % C::kGroups, st = c % C::kStages;
        const uint32_t gp = (uint32_t)(c / C::kGroups) & 1u, cp = (uint32_t)c & 1u;
        const uint32_t kq = tc::smem_u32(smem + st * C::kStageBytes);
        const uint32_t tp = tc::smem_u32(smem + C::kTP + g * C::kTPBytes);
        if (!(ok = tc::mbar_wait(&bars.ready[st], (uint32_t)(c / C::kStages) & 1u))) break;
        if (!(ok = tc::mbar_wait(&bars.s_ready, cp))) break;
        tc::tc_fence_after();
        // X = [K; Q] S
#pragma unroll
        for (int b = 0; b < C::kTiles; ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc::mma_bf16(tmem + kTmX, tc::sw128_desc(kq + (j >> 2) * 16384 + (j & 3) * 32),
                         tc::sw128_desc_mn(s_op + b * 16384 + j * 2048, 0), kIdX, b + j > 0);
        if constexpr (F16) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc::mma_bf16(tmem + kTmX, tc::sw128_desc(kq + 32768 + (j >> 2) * 16384 + (j & 3) * 32),
                         tc::sw128_desc_mn(s_op + j * 2048, 0), kIdX, true);
        }
        tc::mma_commit(&bars.x_full);
        if (!(ok = tc::mbar_wait(&bars.tp_ready[g], gp))) break;
        if (!(ok = tc::mbar_wait(&bars.y_ready, cp))) break;
        tc::tc_fence_after();
        // D = T Y (rows 0..63)
#pragma unroll
        for (int b = 0; b < C::kTiles; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmD, tc::sw128_desc(tp + j * 32), tc::sw128_desc_mn(y_op + b * 8192 + j * 2048, 0), kIdX,
                         b + j > 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tc::mma_bf16(tmem + kTmD, tc::sw128_desc(tp + 16384 + j * 32), tc::sw128_desc_mn(y_op + j * 2048, 0), kIdX, true);
        tc::mma_commit(&bars.d_full);
        if (!(ok = tc::mbar_wait(&bars.u_ready, cp))) break;
        tc::tc_fence_after();
        // dS = K^T D'
#pragma unroll
        for (int b = 0; b < C::kTiles; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmU, tc::sw128_desc_mn(kq + j * 2048, 16384),
                         tc::sw128_desc_mn(y_op + b * 8192 + j * 2048, 0), kIdU, b + j > 0);
        if constexpr (F16) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmU, tc::sw128_desc_mn(kq + 32768 + j * 2048, 16384),
                         tc::sw128_desc_mn(y_op + j * 2048, 0), kIdU, true);
        }
        tc::mma_commit(&bars.u_full);
        tc::mma_commit(&bars.free_[st]);
        if (!(ok = tc::mbar_wait(&bars.v_ready, cp))) break;
        tc::tc_fence_after();
        // P D (rows 64..127)
#pragma unroll
        for (int b = 0; b < C::kTiles; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmO + 64 * (c & 1), tc::sw128_desc(tp + j * 32),
                         tc::sw128_desc_mn(d_op + b * 8192 + j * 2048, 0), kIdX, b + j > 0);
        tc::mma_commit(&bars.o_full[c & 1]);
        tc::mma_commit(&bars.tp_free[g]);
      }
    }
  } else if (warp == C::kMmaWarp + 1) {
    // ------------------------------------------------------------ [K; Q] K^T
    if (lane == 0) {
      constexpr uint32_t kIdA = tc::idesc_bf16_f32(128, 64);
      for (int c = 0; c < nch; ++c) {
        const int st = c % C::kStages;
        const uint32_t kq = tc::smem_u32(smem + st * C::kStageBytes);
        if (!(ok = tc::mbar_wait(&bars.ready[st], (uint32_t)(c / C::kStages) & 1u))) break;
        tc::tc_fence_after();
        const uint32_t d = tmem + kTmA + 64 * (c % C::kGroups);
        const uint32_t lo = kq + 32768;  // FP16: hi hi + hi lo + lo hi
#pragma unroll
        for (int p = 0; p < (F16 ? 3 : 1); ++p)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t off = (j >> 2) * 16384 + (j & 3) * 32;
            tc::mma_bf16(d, tc::sw128_desc((p == 2 ? lo : kq) + off), tc::sw128_desc((p == 1 ? lo : kq) + off), kIdA,
                         p + j > 0);
          }
        tc::mma_commit(&bars.a_full[c % C::kGroups]);
      }
    }
  } else {
    // -------------------------------------------------------------- TMA loads
    if (lane == 0) {
      int issued = 0;
      for (int c = 0; c < nch; ++c) {
        const int st = c % C::kStages;
        if (c >= C::kStages &&
            !(ok = tc::mbar_wait(&bars.free_[st], (uint32_t)(c / C::kStages - 1) & 1u)))
          break;
        uint8_t* kq = smem + st * C::kStageBytes;
        tc::mbar_expect_tx(&bars.full[st], 32768);
        const int tok = (int)t0 + c * kC, hk = h / args.G;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          tma_box(kq + a * 16384, &maps.k, a * 64, hk, tok, &bars.full[st]);
          tma_box(kq + a * 16384 + 8192, &maps.q, a * 64, hk, tok, &bars.full[st]);
        }
        issued = c + 1;
      }
      // nothing may land after the CTA is gone
      for (int c = issued > C::kStages ? issued - C::kStages : 0; c < issued; ++c)
        tc::mbar_wait(&bars.full[c % C::kStages], (uint32_t)(c / C::kStages) & 1u);
    }
  }
  if (!ok) timed_out = 1;
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (tid == 0 && timed_out) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
  if (warp == C::kMmaWarp) tc::tmem_dealloc(tmem, kTmCols);
}

// Tensor map of a [T][heads][128] 16-bit tensor, box (64 elements, 1 head, 64
// tokens) in 128-byte swizzled lines; tokens past the last land as zeros.
bool encode_half_rows(CUtensorMap* m, const void* base, int64_t heads, int64_t T) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t stride[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)heads * kHeadDim * 2};
  const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)kC};
  const cuuint32_t estride[3] = {1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dim, stride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DVS, bool F16>
kda_status launch_prefill(const GdnPrefillArgs& a, const GdnMaps& m, cudaStream_t st) {
  using C = Cfg<DVS, F16>;
  static_assert(C::kSmem + 1024 <= 232448, "shared memory of one CTA");
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_CUDA;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
    if (cudaFuncSetAttribute(gdn_prefill_kernel<DVS, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
        cudaSuccess)
      return KDA_ERR_CUDA;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  const int64_t grid = (int64_t)a.num_seqs * a.HV * (kHeadDim / DVS);
  if (grid > INT32_MAX) return KDA_ERR_SHAPE;
  record_stage(0, st);
  gdn_prefill_kernel<DVS, F16><<<(unsigned)grid, C::kThreads, C::kSmem, st>>>(a, m);
  const kda_status s = launch_status();
  record_stage(1, st);
  record_stage(2, st);
  return s;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_gdn_prefill(kda_dims dims, kda_scalar_gate gate, const kda_bf16* q, const kda_bf16* k,
                                      const kda_bf16* v, const void* a, const kda_bf16* beta, int64_t gb_rows,
                                      float* state_pool, int pool_slots, const int32_t* state_idx,
                                      const int32_t* cu_seqlens, int num_seqs, int64_t total_tokens, kda_bf16* o,
                                      float* intermediate, int64_t intermediate_chunks, int32_t* err_flag,
                                      void* stream) {
  kda_status s = check_dims(dims);
  if (s != KDA_OK) return s;
  if (!state_pool || !state_idx) return KDA_ERR_NULL_ARG;
  if (num_seqs < 0 || pool_slots < 0 || total_tokens < 0 || total_tokens > INT32_MAX || gb_rows < total_tokens)
    return KDA_ERR_SHAPE;
  if (intermediate && intermediate_chunks < 0) return KDA_ERR_SHAPE;
  if (num_seqs == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_SHAPE;
  if (!cu_seqlens && total_tokens % num_seqs != 0) return KDA_ERR_SHAPE;
  if (total_tokens == 0) return KDA_OK;
  if (!q || !k || !v || !a || !beta || !o) return KDA_ERR_NULL_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(state_pool) ||
      !aligned16(intermediate))
    return KDA_ERR_ALIGNMENT;
  GdnPrefillArgs args{};
  s = check_scalar_gate(gate, a, beta, &args.gate);
  if (s != KDA_OK) return s;
  args.H = dims.H;
  args.HV = dims.HV;
  args.G = dims.HV / dims.H;
  args.v = v;
  args.a = a;
  args.beta = beta;
  args.pool = state_pool;
  args.pool_slots = pool_slots;
  args.state_idx = state_idx;
  args.cu_seqlens = cu_seqlens;
  args.num_seqs = num_seqs;
  args.total_tokens = total_tokens;
  args.o = o;
  args.intermediate = intermediate;
  args.inter_chunks = intermediate_chunks;
  args.err_flag = err_flag;
  GdnMaps m;
  if (!encode_half_rows(&m.q, q, dims.H, total_tokens) || !encode_half_rows(&m.k, k, dims.H, total_tokens))
    return KDA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dims.dtype == KDA_DTYPE_F16) return launch_prefill<32, true>(args, m, st);
  const int sms = sm_count();
  if (sms <= 0) return KDA_ERR_CUDA;
  return (int64_t)num_seqs * dims.HV * 4 <= sms ? launch_prefill<32, false>(args, m, st)
                                                : launch_prefill<64, false>(args, m, st);
}
