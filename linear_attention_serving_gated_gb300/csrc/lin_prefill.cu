// lin_prefill.cu -- chunked varlen prefill of linear attention with one decay per
// value head, on tcgen05/TMEM.
//
// Per (sequence, value head), 64 tokens at a time.  c_i is the log-decay summed up
// to token i of the chunk, rq_i and rk_i the inverse norms of its query and key (1
// where they are taken as they are), S (K x V) the state before the chunk:
//   O_i = scale rq_i e^(c_i) (Q S)_i + sum_(j <= i) P_ij v_j,
//         P_ij = scale rq_i rk_j e^(c_i - c_j) q_i.k_j
//   S <- e^(c_last) S + sum_j (e^(c_last - c_j) rk_j k_j) v_j^T
// Decays and norms only scale rows and columns, so the raw 16-bit q and k go into
// Q K^T and Q S as they are, and every exponent is of a difference <= 0.
//
// A CTA takes a segment of a sequence for one value head, all 128 value columns,
// its state in FP32 registers.  Every product but Q K^T is transposed, so that its
// rows are the value columns:
//   Q K^T             64 x 64 x 128
//   O1^T = S^T Q^T   128 x 64 x 128, S^T a left operand from TMEM, in two halves
//   O2^T = V^T P^T   128 x 64 x 64, V as it landed, P in two halves
//   dS^T = V^T K'    128 x 128 x 64, K'_j = e^(c_last - c_j) rk_j k_j in three parts
//                    (FP16: two)
// 8 warps keep the state and turn it into the operand S^T; 4 prepare the chunk's
// factors and K'; 4 turn Q K^T into P and write the outputs; one loads rows, two
// issue the products, those of the state apart from those within the chunk, so
// that neither waits for the other's operands.
//
// A long sequence is cut into segments: a first launch computes what each segment
// adds to a state of zero (no queries, no outputs), and the CTAs of the second sum
// up the state that they start from.  The first segment starts from the pool's state
// in both.
//
// Precision: BF16 halves hi + lo leave 2^-18, three parts 2^-26, FP16 halves 2^-23
// (their range is kept by a power of two for each row of P and of S^T), so that the
// state is as exact as FP32 sums leave it and an output is off by its own rounding.
#include <atomic>

#include "kda_host.h"
#include "kda_tc.cuh"
#include "lin.cuh"

namespace kda {
namespace {

constexpr int kC = 64;  // tokens per chunk
constexpr int kStages = 3, kScalarBufs = 4;

struct LinPrefillArgs {
  LinGateArgs gate;
  int HV, G;
  float* pool;
  int pool_slots;
  const int32_t* state_idx;
  const int32_t* cu_seqlens;
  int num_seqs;
  int64_t total_tokens;
  kda_bf16* o;
  int64_t seg_tokens;   // tokens of a segment, a multiple of 64
  float4* local_state;  // [segment, value head][16][256 threads]: what a segment adds
  float* local_decay;   // [segment, value head]: e^(its log-decays' sum)
  int32_t* err_flag;
};

struct LinMaps {
  CUtensorMap q, k, v;
};

// Factors of a chunk.
struct Scalars {
  float out[kC];      // scale rq_i e^(c_i)
  float row[kC];      // scale rq_i e^(c_i - c_b), b the first token of i's block of 16
  float col[3][kC];   // rk_j e^(c_b - c_j) for b = 16, 32, 48 and j < b
  float q[kC], k[kC]; // scale rq_i, rk_j
  float c_hi[kC], c_lo[kC];
  float last;         // e^(c_last)
  float pad[3];
};

struct Bars {
  uint64_t full[kStages], empty[kStages];  // rows landed, consumed
  uint64_t sc_full[kScalarBufs];           // factors (and V's rows past the end zeroed)
  uint64_t wk_full;                        // K'
  uint64_t ds_full[2], ds_read[2];         // dS
  uint64_t s_full, qs_full;                // operand S^T, O1
  uint64_t qk_full, p_full, o_full;        // Q K^T, P, O2
  uint64_t o_read;                         // O1 and O2 are in registers
  uint64_t drained[2];                     // all products of an issuing warp; used where a wait has run out
  uint32_t tmem;
  int timed_out;
  float p_scale[kC];        // FP16: the powers of two of P's rows
  float s_max[2][2][128];   //       largest magnitudes of half a row of S^T
  float s_scale[2][128];    //       powers of two of its rows
};

// Warps.
constexpr int kStateWarps = 8, kPrepWarp = 8, kOutWarp = 12, kRowWarp = 16, kStateMma = 17, kChunkMma = 18, kSpare = 19,
              kThreads = 640;

// Shared memory: stages of Q, K and V (two halves of 64 channels and 64 lines each),
// the parts of K', P's halves, factors, barriers.
constexpr int kTile = 16384, kStageBytes = 3 * kTile;
constexpr int kWk = kStages * kStageBytes, kP = kWk + 3 * kTile, kScalars = kP + 16384;
constexpr int kBars = kScalars + kScalarBufs * (int)sizeof(Scalars);
constexpr int kSmem = kBars + (int)sizeof(Bars);
static_assert(kSmem <= 232448 - 1024 && kBars % 16 == 0, "shared memory");

// TMEM columns: dS twice, the operand S^T (two 16-bit numbers a column), O1, and
// Q K^T, whose place O2 takes.
constexpr int kTmU = 0, kTmS = 256, kTmSlo = 320, kTmQ = 384, kTmO = 448, kTmCols = 512;

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
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity & 1u));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Two FP32 values as 16-bit numbers, and what is left of them.
template <bool F16>
__device__ __forceinline__ uint32_t round2(float2 x, float2& rest) {
  uint32_t w;
  float2 back;
  if constexpr (F16) {
    const __half2 b = __floats2half2_rn(x.x, x.y);
    w = *reinterpret_cast<const uint32_t*>(&b);
    back = __half22float2(b);
  } else {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
    w = *reinterpret_cast<const uint32_t*>(&b);
    back = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  rest = fma2(back, make_float2(-1.f, -1.f), x);
  return w;
}
template <bool F16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (F16)
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 16-byte piece `piece` of 128-byte line `row` of a 128-byte-swizzled tile.
__device__ __forceinline__ uint4* line16(uint8_t* tile, int row, int piece) {
  return reinterpret_cast<uint4*>(tile + row * 128 + ((piece ^ (row & 7)) << 4));
}

// Waits for this thread's TMEM loads; r is not used before.
template <int M>
__device__ __forceinline__ void wait_ld(uint32_t (&r)[M]) {
  tc::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < M; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_ld8_async(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// 16 rows and 8 columns in the fragment layout: rows lane / 4 and + 8, columns
// 2 (lane % 4) and + 1.
__device__ __forceinline__ void ld_frag8(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem]^T, issued by one thread; 16 k are 8 columns of A.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

__device__ __forceinline__ int64_t seq_start(const LinPrefillArgs& a, int n) {
  return a.cu_seqlens ? (int64_t)a.cu_seqlens[n] : a.total_tokens / a.num_seqs * n;
}
// Tokens of sequence n, -1 where its bounds are not those of a sequence.
__device__ __forceinline__ int seq_len(const LinPrefillArgs& a, int n) {
  const int64_t t0 = seq_start(a, n), t1 = seq_start(a, n + 1);
  const bool bad = t0 < 0 || t1 < t0 || t1 > a.total_tokens || (n == 0 && t0 != 0) ||
                   (n == a.num_seqs - 1 && t1 != a.total_tokens);
  return bad ? -1 : (int)(t1 - t0);
}
__device__ __forceinline__ int seq_segments(const LinPrefillArgs& a, int n) {
  const int len = seq_len(a, n);
  return len > 0 ? (int)((len + a.seg_tokens - 1) / a.seg_tokens) : 0;
}

// The sequence n of segment `id`, and which of its segments it is; n = -1: none.
// Every warp walks over the sequences, 128 at a time.
struct Segment {
  int n, s;
};
__device__ __forceinline__ Segment find_segment(const LinPrefillArgs& args, int id, int lane) {
  Segment r{-1, 0};
  for (int n0 = 0, base = 0; n0 < args.num_seqs && r.n < 0; n0 += 128) {
    int cnt[4], sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = n0 + 4 * lane + e;
      cnt[e] = m < args.num_seqs ? seq_segments(args, m) : 0;
      sum += cnt[e];
    }
    int run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, base + run > id);
    if (past) {
      int at = base + run - sum, mine = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (mine < 0 && id < at + cnt[e]) mine = e;
        if (mine < 0) at += cnt[e];
      }
      const int src = __ffs(past) - 1;
      r.n = n0 + 4 * src + __shfl_sync(0xffffffffu, mine, src);
      r.s = id - __shfl_sync(0xffffffffu, at, src);
    }
    base += __shfl_sync(0xffffffffu, run, 31);
  }
  return r;
}

// Sums of log-decays as pairs hi + lo (two-sum): their differences count.
__device__ __forceinline__ float2 pair_add(float2 a, float2 b) {
  const float s = a.x + b.x, z = s - a.x;
  return make_float2(s, a.y + (((a.x - (s - z)) + (b.x - z)) + b.y));
}
__device__ __forceinline__ float2 pair_from(float2 x, int l) {
  return make_float2(__shfl_sync(0xffffffffu, x.x, l), __shfl_sync(0xffffffffu, x.y, l));
}
__device__ __forceinline__ float exp_diff(float2 a, float2 b) { return expf((a.x - b.x) + (a.y - b.y)); }

// LOCAL: what segments add to a state of zero, or to the pool's.  Otherwise the outputs, and the
// final states.
template <bool F16, bool LOCAL>
__global__ void __launch_bounds__(kThreads, 1)
    lin_prefill_kernel(const LinPrefillArgs args, const __grid_constant__ LinMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + kBars);
  Scalars* scalars = reinterpret_cast<Scalars*>(smem + kScalars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (LOCAL) grid_dependency_launch();
  const int HV = args.HV, h = blockIdx.x % HV, id = blockIdx.x / HV;
  const Segment seg = find_segment(args, id, lane);
  if (!LOCAL && blockIdx.x == 0 && warp == kSpare)  // bounds of no sequence, which has no CTA of its own
    for (int m = lane; m < args.num_seqs; m += 32)
      if (seq_len(args, m) < 0) set_error(args.err_flag, KDA_DEVERR_SEQLENS);
  // whoever waits for the second launch waits for the first one too
  auto leave = [] {
    if (!LOCAL) grid_dependency_wait();
  };
  if (seg.n < 0) {  // the grid is an upper bound
    leave();
    return;
  }
  const int len = seq_len(args, seg.n);
  const int64_t first = (int64_t)seg.s * args.seg_tokens;
  const bool last_segment = first + args.seg_tokens >= len;
  const int L = (int)(last_segment ? len - first : args.seg_tokens), nch = (L + kC - 1) / kC;
  const int64_t t0 = seq_start(args, seg.n) + first;
  const int slot = args.state_idx[seg.n];
  const bool no_slot = slot < 0 || slot >= args.pool_slots;
  if (LOCAL && (last_segment || no_slot)) return;  // nothing starts from its state
  if (no_slot) {  // padding or out of range: zero outputs, no state touched
    if (slot != -1 && tid == 0 && h == 0 && seg.s == 0) set_error(args.err_flag, KDA_DEVERR_SLOT);
    for (int64_t i = tid; i < (int64_t)L * 16; i += kThreads)
      *reinterpret_cast<uint4*>(args.o + ((t0 + i / 16) * HV + h) * kHeadDim + (i % 16) * 8) = make_uint4(0, 0, 0, 0);
    leave();
    return;
  }
  if (tc::smem_u32(smem) & 1023u) {  // swizzled tiles start on 1024 bytes
    if (tid == 0) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
    leave();
    return;
  }
  if (warp == kStateMma) tc::tmem_alloc(&bars.tmem, kTmCols);
  if (tid == 0) {
    bars.timed_out = 0;
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&bars.full[i], 1);
      tc::mbar_init(&bars.empty[i], LOCAL ? 1 : 2);
    }
    for (int i = 0; i < kScalarBufs; ++i) tc::mbar_init(&bars.sc_full[i], 4);
    tc::mbar_init(&bars.wk_full, 4);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.ds_full[i], 1);
      tc::mbar_init(&bars.ds_read[i], kStateWarps);
      tc::mbar_init(&bars.drained[i], 1);
    }
    tc::mbar_init(&bars.s_full, kStateWarps);
    tc::mbar_init(&bars.qs_full, 1);
    tc::mbar_init(&bars.qk_full, 1);
    tc::mbar_init(&bars.p_full, 4);
    tc::mbar_init(&bars.o_full, 1);
    tc::mbar_init(&bars.o_read, 4);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = bars.tmem;
  const LinGateArgs& ga = args.gate;
  // FP16: unit keys are at most 1 and become K' times 2^15, so that small ones keep their places
  const float k_up = F16 && ga.use_qk_l2norm ? 32768.f : 1.f;
  bool ok = true;

  // 640 threads start with 96 registers each; 256 at 128 and 384 at 72 are 60416 of those 61440
  if (warp < kStateWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    // ------------------------------------------------------------------- state
    const int quad = warp & 3, half = warp >> 2;
    const int dv = 32 * quad + lane;  // this thread's value column; its key channels 64 half ..
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    float* root = args.pool + (((size_t)slot * HV + h) * kHeadDim + dv) * kHeadDim + 64 * half;
    float S[64];
    auto record = [&](int64_t segment) { return args.local_state + (segment * HV + h) * 4096 + tid; };
    const int segments = seq_segments(args, seg.n);
    if (!LOCAL) grid_dependency_wait();
    if (seg.s == 0) {
      // The CTA of the last segment writes the sequence's slot, maybe before this one
      // reads it: the first launch leaves a copy where the last segment has no record.
      const bool copied = !LOCAL && segments > 1;
      const float4* copy = record(id + segments - 1);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float4 x = copied ? __ldcg(copy + j * 256) : *reinterpret_cast<const float4*>(root + 4 * j);
        S[4 * j] = x.x, S[4 * j + 1] = x.y, S[4 * j + 2] = x.z, S[4 * j + 3] = x.w;
        if (LOCAL) const_cast<float4*>(copy)[j * 256] = x;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 64; ++j) S[j] = 0.f;
    }
    if (!LOCAL && seg.s > 0) {
      float up = 1.f;  // decay from the end of a segment before to the start of this one
      for (int m = seg.s - 1; m >= 0 && up > 0.f; --m) {
        const float4* src = record(id - seg.s + m);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float4 x = __ldcg(src + j * 256);
          S[4 * j] = fmaf(up, x.x, S[4 * j]);
          S[4 * j + 1] = fmaf(up, x.y, S[4 * j + 1]);
          S[4 * j + 2] = fmaf(up, x.z, S[4 * j + 2]);
          S[4 * j + 3] = fmaf(up, x.w, S[4 * j + 3]);
        }
        up *= __ldcg(args.local_decay + (int64_t)(id - seg.s + m) * HV + h);
      }
    }
    float decay = 1.f;
    const float k_down = 1.f / k_up;
    // A warp that runs out of time goes on without waiting, so that the others still
    // meet it at their barrier.
    for (int c = 0; c < nch; ++c) {
      if (!LOCAL) {
        float down = 1.f, row_scale = 1.f;
        if constexpr (F16) {  // the row relative to its largest, by a power of two
          float m = 0.f;
#pragma unroll
          for (int j = 0; j < 64; ++j) m = fmaxf(m, fabsf(S[j]));
          bars.s_max[c & 1][half][dv] = m;
          asm volatile("barrier.cta.sync 1, 256;" ::: "memory");
          m = fmaxf(m, bars.s_max[c & 1][half ^ 1][dv]);
          uint32_t e = __float_as_uint(m) >> 23;
          e = e < 1 ? 127 : e > 253 ? 253 : e;
          down = __uint_as_float((254u - e) << 23);
          row_scale = __uint_as_float(e << 23);
        }
        if (c > 0) ok = ok && warp_wait(&bars.qs_full, c - 1);  // the operand has been read
        // (and the scales of chunk c - 2, before whose outputs were read Q S of c - 1 did not start)
        if (F16 && half == 0) bars.s_scale[c & 1][dv] = row_scale;
        tc::tc_fence_after();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float2 x = make_float2(S[16 * g + 2 * j], S[16 * g + 2 * j + 1]), rest;
            if (F16) x = mul2(x, make_float2(down, down));
            hi[j] = round2<F16>(x, rest);
            lo[j] = round2<F16>(rest, x);
          }
          tmem_st8(lanes + kTmS + 32 * half + 8 * g, hi);
          tmem_st8(lanes + kTmSlo + 32 * half + 8 * g, lo);
        }
        wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) arrive(&bars.s_full);
        if (c == nch - 1 && !last_segment) break;  // its state is of no use
      }
      ok = ok && warp_wait(&bars.sc_full[c % kScalarBufs], c / kScalarBufs);
      const float last = scalars[c % kScalarBufs].last;
      ok = ok && warp_wait(&bars.ds_full[c & 1], c >> 1);
      tc::tc_fence_after();
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t r[16];
        tc::tmem_ld16_async(lanes + kTmU + 128 * (c & 1) + 64 * half + 16 * g, r);
        wait_ld(r);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          float2 u = make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1]));
          if (F16) u = mul2(u, make_float2(k_down, k_down));
          const float2 s = fma2(make_float2(last, last), make_float2(S[16 * g + j], S[16 * g + j + 1]), u);
          S[16 * g + j] = s.x;
          S[16 * g + j + 1] = s.y;
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) arrive(&bars.ds_read[c & 1]);
      decay *= last;
    }
    if (LOCAL) {
      float4* dst = record(id);
#pragma unroll
      for (int j = 0; j < 16; ++j) dst[j * 256] = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
      if (tid == 0) args.local_decay[(int64_t)id * HV + h] = decay;
    } else if (ok && last_segment) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        *reinterpret_cast<float4*>(root + 4 * j) = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp < kOutWarp) {
      // ------------------------------------------------- a chunk's factors and K'
      const int w = warp - kPrepWarp, row = 16 * w + (lane & 15), half = lane >> 4;
      const float neg_rate = ga.A_log ? -expf(ga.A_log[h]) : 0.f;
      const float bias = ga.dt_bias ? ga.dt_bias[h] : 0.f;
      ushort2 raw[2];
      auto load_gate = [&](int c) {  // tokens 2 lane and 2 lane + 1
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          raw[e] = make_ushort2(0, 0);
          if (c * kC + 2 * lane + e < L) raw[e] = lin_gate_load(ga, (t0 + c * kC + 2 * lane + e) * HV + h);
        }
      };
      load_gate(0);
      for (int c = 0; c < nch; ++c) {
        const int st = c % kStages, left = L - c * kC;
        Scalars& sc = scalars[c % kScalarBufs];
        float2 even, run;  // c of tokens 2 lane, 2 lane + 1
        {
          const float g0 = 2 * lane < left ? lin_log_decay<F16>(ga, raw[0], neg_rate, bias) : 0.f;
          const float g1 = 2 * lane + 1 < left ? lin_log_decay<F16>(ga, raw[1], neg_rate, bias) : 0.f;
          run = pair_add(make_float2(g0, 0.f), make_float2(g1, 0.f));
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const float2 up = make_float2(__shfl_up_sync(0xffffffffu, run.x, d), __shfl_up_sync(0xffffffffu, run.y, d));
            if (lane >= d) run = pair_add(up, run);
          }
          even = pair_add(run, make_float2(-g1, 0.f));
        }
        if (c + 1 < nch) load_gate(c + 1);
        const float2 c_last = pair_from(run, 31);
        const float2 a = pair_from(even, row >> 1), b = pair_from(run, row >> 1);
        const float2 c_i = row & 1 ? b : a;
        const float2 c_b = pair_from(even, 8 * w);
        if (!(ok = warp_wait(&bars.full[st], c / kStages))) break;
        uint8_t* rows = smem + st * kStageBytes;
        uint4 kw[8];
        float2 sk = make_float2(0.f, 0.f), sq = make_float2(0.f, 0.f);
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          kw[p] = *line16(rows + kTile + half * 8192, row, p);
          const uint32_t x[4] = {kw[p].x, kw[p].y, kw[p].z, kw[p].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = widen2<F16>(x[e]);
            sk = fma2(f, f, sk);
          }
        }
        if (!LOCAL) {
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const uint4 qw = *line16(rows + half * 8192, row, p);
            const uint32_t x[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = widen2<F16>(x[e]);
              sq = fma2(f, f, sq);
            }
          }
        }
        float nk = sk.x + sk.y, nq = sq.x + sq.y;
        nk += __shfl_xor_sync(0xffffffffu, nk, 16);
        nq += __shfl_xor_sync(0xffffffffu, nq, 16);
        const float rk = ga.use_qk_l2norm ? rsqrtf(nk + kNormEps) : 1.f;
        const float rq = ga.scale * (ga.use_qk_l2norm ? rsqrtf(nq + kNormEps) : 1.f);
        if (half == 0) {
          sc.out[row] = rq * expf(c_i.x + c_i.y);
          sc.row[row] = rq * exp_diff(c_i, c_b);
          sc.q[row] = rq;
          sc.k[row] = rk;
          sc.c_hi[row] = c_i.x;
          sc.c_lo[row] = c_i.y;
          if (row == 0) sc.last = expf(c_last.x + c_last.y);
        }
        if (!LOCAL)
          for (int x = 1; x < 4; ++x) {  // every lane takes part in the exchange
            const float2 ref = pair_from(even, 8 * x);
            if (x > w && (x & 1) == half) sc.col[x - 1][row] = rk * exp_diff(ref, c_i);
          }
        if (left < kC && row >= left) {  // the next sequence's values: NaN times zero is NaN
#pragma unroll
          for (int p = 0; p < 8; ++p) *line16(rows + 2 * kTile + half * 8192, row, p) = make_uint4(0, 0, 0, 0);
          tc::fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) arrive(&bars.sc_full[c % kScalarBufs]);
        const float wk = row < left ? k_up * rk * exp_diff(c_last, c_i) : 0.f;
        if (c > 0 && !(ok = warp_wait(&bars.ds_full[(c - 1) & 1], (c - 1) >> 1))) break;  // K' has been read
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const uint32_t x[4] = {kw[p].x, kw[p].y, kw[p].z, kw[p].w};
          uint32_t part[3][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 f = mul2(widen2<F16>(x[e]), make_float2(wk, wk)), rest;
            if (row >= left) f = make_float2(0.f, 0.f);
            part[0][e] = round2<F16>(f, rest);
            part[1][e] = round2<F16>(rest, f);
            if (!F16) part[2][e] = round2<F16>(f, rest);
          }
#pragma unroll
          for (int i = 0; i < (F16 ? 2 : 3); ++i)
            *line16(smem + kWk + i * kTile + half * 8192, row, p) = make_uint4(part[i][0], part[i][1], part[i][2], part[i][3]);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive(&bars.wk_full);
      }
    } else if (warp < kRowWarp) {
      // ---------------------------------------------------------- P, and the outputs
      if (!LOCAL) {
        const int w = warp - kOutWarp, r0 = 16 * w + (lane >> 2);  // rows r0 and r0 + 8
        const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
        const int odd = lane & 1;
        const uint32_t pick = odd ? 0x3276u : 0x5410u;
        const int64_t step = (int64_t)HV * kHeadDim;
        kda_bf16* dst = args.o + ((t0 + odd) * HV + h) * kHeadDim + ((32 * w + lane) & ~1);
        for (int c = 0; c < nch; ++c, dst += kC * step) {
          const Scalars& sc = scalars[c % kScalarBufs];
          if (!(ok = warp_wait(&bars.sc_full[c % kScalarBufs], c / kScalarBufs))) break;
          const float fr[2] = {sc.row[r0], sc.row[r0 + 8]}, fq[2] = {sc.q[r0], sc.q[r0 + 8]};
          const float ch[2] = {sc.c_hi[r0], sc.c_hi[r0 + 8]}, cl[2] = {sc.c_lo[r0], sc.c_lo[r0 + 8]};
          if (!(ok = warp_wait(&bars.qk_full, c))) break;
          tc::tc_fence_after();
          float2 p[8][2];
          uint32_t r[4][4];
          float big[2] = {0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j % 4 == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) ld_frag8(lanes + kTmO + 8 * (j + i), r[i]);
#pragma unroll
              for (int i = 0; i < 4; ++i) wait_ld(r[i]);
            }
            const int col = 8 * j + 2 * (lane & 3);
            float f[2][2];  // the factors of rows r0, r0 + 8 and columns col, col + 1
            if (j < 2 * w) {
              const float2 x = *reinterpret_cast<const float2*>(&sc.col[w - 1][col]);
              f[0][0] = fr[0] * x.x, f[0][1] = fr[0] * x.y, f[1][0] = fr[1] * x.x, f[1][1] = fr[1] * x.y;
            } else if (j < 2 * w + 2) {
              const float2 k2 = *reinterpret_cast<const float2*>(&sc.k[col]), h2 = *reinterpret_cast<const float2*>(&sc.c_hi[col]),
                           l2 = *reinterpret_cast<const float2*>(&sc.c_lo[col]);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                f[e][0] = fq[e] * k2.x * __expf(fminf((ch[e] - h2.x) + (cl[e] - l2.x), 0.f));
                f[e][1] = fq[e] * k2.y * __expf(fminf((ch[e] - h2.y) + (cl[e] - l2.y), 0.f));
              }
            } else {
              f[0][0] = f[0][1] = f[1][0] = f[1][1] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = r0 + 8 * e;
              p[j][e].x = col <= i ? f[e][0] * __uint_as_float(r[j % 4][2 * e]) : 0.f;
              p[j][e].y = col + 1 <= i ? f[e][1] * __uint_as_float(r[j % 4][2 * e + 1]) : 0.f;
              if (F16) big[e] = fmaxf(big[e], fmaxf(fabsf(p[j][e].x), fabsf(p[j][e].y)));
            }
          }
          float down[2] = {1.f, 1.f};
          if constexpr (F16) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              big[e] = fmaxf(big[e], __shfl_xor_sync(0xffffffffu, big[e], 1));
              big[e] = fmaxf(big[e], __shfl_xor_sync(0xffffffffu, big[e], 2));
              uint32_t x = __float_as_uint(big[e]) >> 23;
              x = x < 1 ? 127 : x > 253 ? 253 : x;
              down[e] = __uint_as_float((254u - x) << 23);
              if ((lane & 3) == 0) bars.p_scale[r0 + 8 * e] = __uint_as_float(x << 23);
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = r0 + 8 * e;
              float2 x = p[j][e], rest;
              if (F16) x = mul2(x, make_float2(down[e], down[e]));
              const uint32_t hi = round2<F16>(x, rest), lo = round2<F16>(rest, x);
              const int at = i * 128 + ((j ^ (i & 7)) << 4) + 4 * (lane & 3);
              *reinterpret_cast<uint32_t*>(smem + kP + at) = hi;
              *reinterpret_cast<uint32_t*>(smem + kP + 8192 + at) = lo;
            }
          tc::fence_async_smem();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive(&bars.p_full);
          // outputs: 32 value columns a warp, 64 tokens a thread
          if (!(ok = warp_wait(&bars.qs_full, c) && warp_wait(&bars.o_full, c))) break;
          tc::tc_fence_after();
          const float up = F16 ? bars.s_scale[c & 1][32 * w + lane] : 1.f;
          const int left = L - c * kC - odd;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint32_t y2[16];  // two tokens of one column each
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const int tok = 32 * part + 8 * g;
              uint32_t q[8], r[8];
              tmem_ld8_async(lanes + kTmQ + tok, q);
              tmem_ld8_async(lanes + kTmO + tok, r);
              wait_ld(q);
              wait_ld(r);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float2 f = *reinterpret_cast<const float2*>(sc.out + tok + 2 * j);
                float2 y = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                if (F16) {
                  f = mul2(f, make_float2(up, up));
                  y = mul2(y, *reinterpret_cast<const float2*>(bars.p_scale + tok + 2 * j));
                }
                y = fma2(f, make_float2(__uint_as_float(q[2 * j]), __uint_as_float(q[2 * j + 1])), y);
                y2[4 * g + j] = pack_out16x2<F16>(y.x, y.y);
              }
            }
            if (part) {
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive(&bars.o_read);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {  // traded for two columns of one token each
              const int tok = 32 * part + 2 * j;
              const uint32_t x = __byte_perm(y2[j], __shfl_xor_sync(0xffffffffu, y2[j], 1), pick);
              if (tok < left) *reinterpret_cast<uint32_t*>(dst + tok * step) = x;
            }
          }
        }
      }
    } else if (warp == kRowWarp) {
      // -------------------------------------------------------------------- rows
      const bool leader = elect_one();
      int issued = 0;
      for (int c = 0; c < nch; ++c) {
        const int st = c % kStages;
        if (c >= kStages && !(ok = warp_wait(&bars.empty[st], c / kStages - 1))) break;
        uint8_t* rows = smem + st * kStageBytes;
        if (leader) {
          tc::mbar_expect_tx(&bars.full[st], LOCAL ? 2 * kTile : kStageBytes);
          const int tok = (int)t0 + c * kC;
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            tma_box(rows + kTile + a * 8192, &maps.k, a * 64, h / args.G, tok, &bars.full[st]);
            if (!LOCAL) tma_box(rows + a * 8192, &maps.q, a * 64, h / args.G, tok, &bars.full[st]);
            tma_box(rows + 2 * kTile + a * 8192, &maps.v, a * 64, h, tok, &bars.full[st]);
          }
        }
        __syncwarp();
        issued = c + 1;
      }
      // nothing may land after the CTA is gone
      for (int c = issued > kStages ? issued - kStages : 0; c < issued; ++c) warp_wait(&bars.full[c % kStages], c / kStages);
    } else if (warp == kStateMma) {
      // ------------------------------------------------- products of the state
      constexpr uint32_t kType = F16 ? tc::idesc_f16_f32(128, 64) : tc::idesc_bf16_f32(128, 64);
      constexpr uint32_t kIdU = (F16 ? tc::idesc_f16_f32(128, 128) : tc::idesc_bf16_f32(128, 128)) | tc::kIdescMnA | tc::kIdescMnB;
      const bool leader = elect_one();
      const uint64_t wk_op = tc::sw128_desc_mn(tc::smem_u32(smem + kWk), 8192);
      for (int c = 0; c < nch; ++c) {
        const int st = c % kStages;
        const uint32_t rows = tc::smem_u32(smem + st * kStageBytes);
        const uint64_t q_op = tc::sw128_desc(rows), v_op = tc::sw128_desc_mn(rows + 2 * kTile, 8192);
        if (!(ok = warp_wait(&bars.full[st], c / kStages) && warp_wait(&bars.wk_full, c))) break;
        if (c > 1 && !(ok = warp_wait(&bars.ds_read[c & 1], (c >> 1) - 1))) break;
        tc::tc_fence_after();
        if (leader) {  // dS^T = V^T K'
#pragma unroll
          for (int b = 0; b < (F16 ? 2 : 3); ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tc::mma_bf16(tmem + kTmU + 128 * (c & 1), v_op + ((j * 2048) >> 4), wk_op + ((b * kTile + j * 2048) >> 4), kIdU,
                           b + j > 0);
          tc::mma_commit(&bars.ds_full[c & 1]);
          if (LOCAL) tc::mma_commit(&bars.empty[st]);
        }
        __syncwarp();
        if (!LOCAL) {
          if (!(ok = warp_wait(&bars.s_full, c))) break;
          if (c > 0 && !(ok = warp_wait(&bars.o_read, c - 1))) break;
          tc::tc_fence_after();
          if (leader) {  // O1^T = S^T Q^T
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int j = 0; j < 8; ++j)
                mma_ts(tmem + kTmQ, tmem + (b ? kTmSlo : kTmS) + 8 * j, q_op + (((j >> 2) * 8192 + (j & 3) * 32) >> 4), kType,
                       b + j > 0);
            tc::mma_commit(&bars.qs_full);
            tc::mma_commit(&bars.empty[st]);
          }
          __syncwarp();
        }
      }
    } else if (warp == kChunkMma) {
      // -------------------------------------------- products within the chunk
      if (!LOCAL) {
        constexpr uint32_t kIdP = F16 ? tc::idesc_f16_f32(64, 64) : tc::idesc_bf16_f32(64, 64);
        constexpr uint32_t kIdO = (F16 ? tc::idesc_f16_f32(128, 64) : tc::idesc_bf16_f32(128, 64)) | tc::kIdescMnA;
        const bool leader = elect_one();
        const uint64_t p_op = tc::sw128_desc(tc::smem_u32(smem + kP));
        for (int c = 0; c < nch; ++c) {
          const int st = c % kStages;
          const uint32_t rows = tc::smem_u32(smem + st * kStageBytes);
          const uint64_t q_op = tc::sw128_desc(rows), k_op = tc::sw128_desc(rows + kTile);
          const uint64_t v_op = tc::sw128_desc_mn(rows + 2 * kTile, 8192);
          if (!(ok = warp_wait(&bars.full[st], c / kStages))) break;
          if (c > 0 && !(ok = warp_wait(&bars.o_read, c - 1))) break;  // Q K^T takes the place of the last O2
          tc::tc_fence_after();
          if (leader) {  // Q K^T
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint64_t off = ((j >> 2) * 8192 + (j & 3) * 32) >> 4;
              tc::mma_bf16(tmem + kTmO, q_op + off, k_op + off, kIdP, j > 0);
            }
            tc::mma_commit(&bars.qk_full);
          }
          __syncwarp();
          if (!(ok = warp_wait(&bars.p_full, c))) break;
          tc::tc_fence_after();
          if (leader) {  // O2^T = V^T P^T
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tc::mma_bf16(tmem + kTmO, v_op + ((j * 2048) >> 4), p_op + ((b * 8192 + j * 32) >> 4), kIdO, b + j > 0);
            tc::mma_commit(&bars.o_full);
            tc::mma_commit(&bars.empty[st]);
          }
          __syncwarp();
        }
      }
    }
  }
  // Where a wait has run out, products may still be under way: their issuing warps
  // wait for them, with a limit, before TMEM and shared memory go.
  if (!ok) bars.timed_out = 1;
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (bars.timed_out) {
    if (tid == 0) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
    if (warp == kStateMma || warp == kChunkMma) {
      uint64_t* bar = &bars.drained[warp == kChunkMma];
      if (elect_one()) tc::mma_commit(bar);  // the same lane as issued them
      __syncwarp();
      warp_wait(bar, 0);
    }
    __syncthreads();
  } else {
    // every product has been waited for but the last ones whose results nobody needs
    if (warp == kStateMma) {
      if (elect_one()) tc::mma_commit(&bars.drained[0]);
      __syncwarp();
      warp_wait(&bars.drained[0], 0);
    }
    __syncthreads();
  }
  if (warp == kStateMma) tc::tmem_dealloc(tmem, kTmCols);
}

// Tensor map of a [T][heads][128] 16-bit tensor, box (64 elements, 1 head, 64
// tokens) in 128-byte swizzled lines; tokens past the last land as zeros.
bool encode_rows(CUtensorMap* m, const void* base, int64_t heads, int64_t T) {
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

// The kernels' shared-memory limits, all of them in the first call on a device: a
// later one may be under capture.
kda_status allow_all() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_CUDA;
  if (ready.load(std::memory_order_relaxed) >> dev & 1u) return KDA_OK;
  auto allow = [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess;
  };
  if (!allow(lin_prefill_kernel<false, false>) || !allow(lin_prefill_kernel<false, true>) ||
      !allow(lin_prefill_kernel<true, false>) || !allow(lin_prefill_kernel<true, true>))
    return KDA_ERR_CUDA;
  ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  return KDA_OK;
}

// Tokens of a segment: so many that all segments of all heads fill the SMs about
// once, 256 at least.
constexpr int64_t kSms = 152;
int64_t segment_tokens(const kda_dims& d, int64_t total_tokens) {
  const int64_t even = (total_tokens * d.HV + kSms - 1) / kSms;
  const int64_t L = (even + kC - 1) / kC * kC;
  return L < 256 ? 256 : L;
}
int64_t most_segments(const kda_dims& d, int num_seqs, int64_t total_tokens) {
  return total_tokens / segment_tokens(d, total_tokens) + num_seqs;
}

}  // namespace
}  // namespace kda

using namespace kda;

// A record of what each segment adds, and its decay; none where no sequence can
// have two segments.
extern "C" size_t kda_lin_prefill_workspace_size(kda_dims dims, int num_seqs, int64_t total_tokens) {
  if (num_seqs < 0 || total_tokens < 0 || dims.H <= 0 || dims.HV <= 0) return 0;
  if (total_tokens > INT32_MAX) return SIZE_MAX;  // refused; no capacity check may pass
  if (total_tokens <= segment_tokens(dims, total_tokens)) return 0;
  return (size_t)most_segments(dims, num_seqs, total_tokens) * dims.HV * (65536 + 16);
}

extern "C" kda_status kda_lin_prefill(kda_dims dims, kda_scalar_gate gate, const kda_bf16* q, const kda_bf16* k,
                                      const kda_bf16* v, const void* a, int64_t gate_rows, float* state_pool,
                                      int pool_slots, const int32_t* state_idx, const int32_t* cu_seqlens, int num_seqs,
                                      int64_t total_tokens, kda_bf16* o, void* workspace, size_t workspace_bytes,
                                      int32_t* err_flag, void* stream) {
  kda_status s = check_dims(dims);
  if (s != KDA_OK) return s;
  if (!state_pool || !state_idx) return KDA_ERR_NULL_ARG;
  if (num_seqs < 0 || pool_slots < 0 || total_tokens < 0 || total_tokens > INT32_MAX || (a && gate_rows < total_tokens))
    return KDA_ERR_SHAPE;
  if (num_seqs == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_SHAPE;
  if (!cu_seqlens && total_tokens % num_seqs != 0) return KDA_ERR_SHAPE;
  if (total_tokens == 0) return KDA_OK;
  if (!q || !k || !v || !o) return KDA_ERR_NULL_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(state_pool)) return KDA_ERR_ALIGNMENT;
  const size_t need = kda_lin_prefill_workspace_size(dims, num_seqs, total_tokens);
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return KDA_ERR_ALIGNMENT;
  LinPrefillArgs args{};
  s = check_lin_gate(gate, a, &args.gate);
  if (s != KDA_OK) return s;
  args.HV = dims.HV;
  args.G = dims.HV / dims.H;
  args.pool = state_pool;
  args.pool_slots = pool_slots;
  args.state_idx = state_idx;
  args.cu_seqlens = cu_seqlens;
  args.num_seqs = num_seqs;
  args.total_tokens = total_tokens;
  args.o = o;
  args.seg_tokens = segment_tokens(dims, total_tokens);
  args.err_flag = err_flag;
  const int64_t units = most_segments(dims, num_seqs, total_tokens) * dims.HV;
  if (units > INT32_MAX) return KDA_ERR_SHAPE;
  args.local_state = static_cast<float4*>(workspace);
  args.local_decay = reinterpret_cast<float*>(static_cast<char*>(workspace) + (need > 0 ? (size_t)units * 65536 : 0));
  LinMaps m;
  if (!encode_rows(&m.q, q, dims.H, total_tokens) || !encode_rows(&m.k, k, dims.H, total_tokens) ||
      !encode_rows(&m.v, v, dims.HV, total_tokens))
    return KDA_ERR_CUDA;
  s = allow_all();
  if (s != KDA_OK) return s;
  const bool f16 = dims.dtype == KDA_DTYPE_F16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  record_stage(0, st);
  if (need > 0) {
    s = launch_dependent(f16 ? lin_prefill_kernel<true, true> : lin_prefill_kernel<false, true>, (unsigned)units, kThreads, kSmem,
                         false, st, args, m);
    if (s != KDA_OK) return s;
  }
  record_stage(1, st);
  s = launch_dependent(f16 ? lin_prefill_kernel<true, false> : lin_prefill_kernel<false, false>, (unsigned)units, kThreads, kSmem,
                       need > 0 && !stage_between(), st, args, m);
  record_stage(2, st);
  return s;
}
