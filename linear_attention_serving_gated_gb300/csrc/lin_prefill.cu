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
// 16 warps do all the arithmetic, together and a step of it at a time, since what they
// execute then is in the SM's instruction caches: per chunk the state's update and its
// operand, P, the outputs of the chunk before, and K' of the chunk behind.
// (Warps of a task each ran at 6 to 8 cycles an instruction, waiting for it: 5000
// cycles a chunk.)  The products run meanwhile: each has a step or more of other work
// before it is needed.  One warp loads rows, one issues products, two make the factors
// of the decays, four those of the norms.
//
// Bound by the workers' instructions: 4800 cycles a chunk, in the shadow of which are the
// products, and 2200 in the first launch.  1 x 4096 tokens at 16 heads 44 us (69 MB:
// 1.6 TB/s), 8 x 4096 162 us (3.4 TB/s), 16 980 tokens in eight sequences 126 us;
// 1 x 128 at 4 heads 11 us, a third of it a CTA's start.
//
// A long sequence is cut into segments: a first launch computes what each segment
// adds to a state of zero (no queries, no outputs), and the CTAs of the second sum
// up the state that they start from.  The first segment starts from the pool's state
// in both.  (Whole, the 64 chunks of 1 x 4096 would take some 150 us on 16 SMs.)
//
// Precision.  The state is FP32, in registers and in the pool.  K' is split in three
// BF16 parts, 2^-26 of it left, or two FP16 ones, 2^-23 of it or 2^-39 of the chunk's
// largest, so that states are as exact as FP32 sums leave them.  S^T and P as operands
// are halves hi + lo of the outputs' type, 2^-17 (FP16: 2^-23) of them left, so that an
// output is as exact as its own rounding.  (Rounded once, they made outputs up to sqrt 2
// times as far off, for 4 to 9% less time: the second halves' instructions, not their
// products.)  FP16's range is kept by a power of two for each row of P and of S^T, and for
// a chunk's K'.
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
  int pool_slots;
  const int32_t* state_idx;
  const int32_t* cu_seqlens;
  int num_seqs;
  int64_t total_tokens, each;  // tokens; of a sequence, without cu_seqlens
  kda_bf16* o;
  // tokens of a segment, multiples of 64: where no sequence is longer than even_most,
  // and otherwise; sequences of at most uncut tokens then stay in one piece
  int seg_even, seg_ragged, even_most, uncut;
  float4* local_state;  // [segment, value head][8][512 threads]: what a segment adds
  float* local_decay;   // [segment, value head]: e^(its log-decays' sum), negative where that state is not finite
  int32_t* err_flag;
};

struct LinMaps {
  CUtensorMap q, k, v, pool;
};

// Factors of a chunk: of the decays first, then times those of the norms.  c_b is halfway
// between c of the first and of the last token of i's block of 16, so that both factors of a
// weight stay within e^30 (from the first token they reach e^60, and tokens of size 1e6, not
// normalised, FP32's largest); where a block decays by more than e^60 the block's rows of P get
// their factors term by term (far).
struct Scalars {
  float c_hi[kC], c_lo[kC];  // c_i
  float out[kC];             // scale rq_i e^(c_i)
  float row[kC];             // scale rq_i e^(c_i - c_b); far: scale rq_i
  float col[4][kC];          // rk_j e^(c_b - c_j) for the four blocks and j up to their ends
  float w[kC];               // rk_j e^(c_last - c_j), 0 past the segment's end
  float k[kC];               // rk_j
  float big[kC], kk[kC];     // FP16: |q_i| e^(c_b - c_i), far |q_i|; |k_j|^2
  float k_big[4];            // FP16, keys as they are: the largest w_j |k_j| of 16 tokens each
  int far[4];                // of the four blocks
  float last;                // e^(c_last)
  float pad[3];
};
constexpr float kFar = 60.f;

// Warps.  Who waits for whom is run in a model, with the places that are written and read:
// tests/test_lin_handover_cpu.py and tests/test_lin_handover_halves_cpu.py (the second
// launch).  A change of the hand-overs here goes there too.
constexpr int kWorkers = 16, kRowWarp = 16, kMmaWarp = 17, kGateWarp = 18, kNormWarp = 20, kNormWarps = 4, kThreads = 768;

struct Bars {
  uint64_t full[kStages];            // rows landed
  uint64_t empty[kStages];           // and consumed
  uint64_t gate_full[kScalarBufs];   // factors of the decays
  uint64_t in_full[kScalarBufs];     // rows and all factors
  uint64_t sc_free[kScalarBufs];     // factors read
  uint64_t wk_full[2];               // operands: K' (and what else a chunk needs), chunks in turn,
  uint64_t u_full, p_full;           // dS is in registers; S^T and P
  uint64_t ds_full[2];               // products: dS, chunks in turn,
  uint64_t qk_full;                  // Q K^T
  uint64_t o_full;                   // O1 and O2
  uint64_t drained;                  // all products
  uint64_t state_full, state_read;   // the pool's state landed, and is in registers
  uint32_t tmem;
  int timed_out;
  float p_scale[2][kC];      // FP16: the powers of two of P's rows
  float s_scale[3][128];     //       and of S^T's
  uint8_t s_big[2][4][128];  //       exponents of the largest of a quarter of a row
};

// Shared memory: stages of Q, K and V (two halves of 64 channels and 64 lines each),
// the parts of K', P's halves, factors, barriers.  The pool's state lands, in four boxes of
// 32 key channels, where chunk 2's rows (LOCAL: chunk 1's K') and P will be, and leaves the
// same way.  (Plain accesses, 32 bytes a lane and lanes 512 apart, held up the SM's memory
// instructions for 3500 cycles.)
constexpr int kTile = 16384, kStageBytes = 3 * kTile;
constexpr int kWk = kStages * kStageBytes, kP = kWk + 3 * kTile, kScalars = kP + kTile;
constexpr int kLocalStage = 2 * kTile, kLocalWk = 3 * kTile;  // LOCAL: K and V alone, and K' twice
static_assert(kStages * kLocalStage + 2 * kLocalWk <= kScalars, "the first launch's layout");
constexpr int kState = 2 * kStageBytes, kLocalState = kWk;
static_assert(kStages * kLocalStage + kLocalWk == kLocalState, "the second K' of the first launch");
constexpr int kBars = kScalars + kScalarBufs * (int)sizeof(Scalars);
constexpr int kSmem = kBars + (int)sizeof(Bars);
static_assert(kSmem <= 232448 - 1024 && kBars % 16 == 0, "shared memory");

// TMEM columns: dS (the first launch's second one beside it), the halves of the operand S^T
// (two 16-bit numbers a column), and for chunks in turn O1, and Q K^T, whose place O2 takes.
constexpr int kTmU = 0, kTmS = 128, kTmQ = 256, kTmO = 384, kTmCols = 512;

__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store_box(const CUtensorMap* map, int c0, int c1, int c2, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
// A wait of two seconds at most; false: it ran out.
//
// A barrier's phase is known by its parity alone, so that a waiter must not fall two
// phases behind, and who arrives must not be a phase ahead of the others: each phase of
// a barrier here needs arrivals that come after every wait for the phase before last
// and every arrival at the last one.  Where a chunk's alone would not see to that, there
// is a barrier for either parity of the chunk.
__device__ __forceinline__ bool long_wait(uint64_t* bar, uint32_t parity) {
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
  do {
    if (tc::mbar_try_wait(bar, parity)) return true;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  } while (t - t0 < 2000000000ull);
  return false;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t phase) {
  const uint32_t parity = phase & 1u;
  if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, long_wait(bar, parity));
}
// Whether it is so for any thread of the 16 worker warps, which all come here.
__device__ __forceinline__ bool any_worker(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 512, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
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

// The power of two that takes numbers of up to m near FP16's largest, below 2^15,
// where the steps at the other end matter least; and back.
__device__ __forceinline__ float to_2p15(uint32_t x, float& back) {  // x: m's exponent field; m < 2^(x - 126)
  x = x < 15 ? 15 : x > 253 ? 253 : x;
  back = __uint_as_float((x - 14) << 23);
  return __uint_as_float((268 - x) << 23);
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

__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

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
  return a.cu_seqlens ? (int64_t)a.cu_seqlens[n] : a.each * n;
}
// Tokens of sequence n, -1 where its bounds are not those of a sequence.
__device__ __forceinline__ int seq_len(const LinPrefillArgs& a, int n) {
  const int64_t t0 = seq_start(a, n), t1 = seq_start(a, n + 1);
  const bool bad = t0 < 0 || t1 < t0 || t1 > a.total_tokens || (n == 0 && t0 != 0) ||
                   (n == a.num_seqs - 1 && t1 != a.total_tokens);
  return bad ? -1 : (int)(t1 - t0);
}
// A CTA's segment: the s-th of `count` of sequence n (-1: none), `tokens` long but for
// the last; `record` is the place of the sequence's first segment among those of
// sequences in several.
struct Segment {
  int n, s, count, record, tokens;
  int len;     // of the sequence
  int64_t t0;  // its first token
};

// The id-th segment: longer sequences that stay in one piece, then the whole segments of
// the others, then what is left of those and the short ones, so that the longest start
// first; LOCAL: the id-th whole segment.  Every warp finds it for itself, a sequence a lane.
// (What runs once a CTA is kept short: instructions that no cache holds yet take five
// or more times as long as others.)
template <bool LOCAL>
__device__ __forceinline__ Segment find_segment(const LinPrefillArgs& args, int id, int lane) {
  const int seqs = args.num_seqs;
  Segment r{-1, 0, 0, 0, args.seg_even, 0, 0};
  int L = args.seg_even;
  if (seqs == 1) {
    const int len = seq_len(args, 0), count = len > 0 ? (len + L - 1) / L : 0;
    if (id < count) r = Segment{0, id, count, 0, L, len, 0};
    return r;
  }
  int most = 0, uncut = 0;
  int64_t sum = 0;
#pragma unroll 1
  for (int m = lane; m < seqs; m += 32) {
    const int len = max(seq_len(args, m), 0);
    most = max(most, len);
    sum += len;
  }
  most = __reduce_max_sync(0xffffffffu, most);
#pragma unroll 1
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (sum > args.total_tokens) return r;  // they overlap: more segments than there is room for
  if (most > args.even_most) {
    L = args.seg_ragged;
    uncut = args.uncut;
  }
  r.tokens = L;
  int base = 0;
  if (most <= L) {  // every sequence is one segment: the id-th that has tokens
#pragma unroll 1
    for (int n0 = 0; !LOCAL && n0 < seqs; n0 += 32) {
      const int len = n0 + lane < seqs ? seq_len(args, n0 + lane) : 0;
      const unsigned some = __ballot_sync(0xffffffffu, len > 0);
      if (base + __popc(some) > id) {
        const int src = __fns(some, 0, id - base + 1);
        r.n = n0 + src;
        r.len = __shfl_sync(0xffffffffu, len, src);
        r.count = 1;
        r.t0 = seq_start(args, r.n);
        break;
      }
      base += __popc(some);
    }
    return r;
  }
#pragma unroll 1
  for (int turn = LOCAL || !uncut ? 1 : 0; turn < (LOCAL ? 2 : 3) && r.n < 0; ++turn) {
    int records = 0;
#pragma unroll 1
    for (int n0 = 0; n0 < seqs && r.n < 0; n0 += 32) {
      const int m = n0 + lane, len = m < seqs ? max(seq_len(args, m), 0) : 0;
      const bool one = len > L && len <= uncut;
      const int whole = one ? 0 : len / L, all = one ? 1 : whole + (len != whole * L);
      const int mine = turn == 0 ? one : turn == 1 ? whole : one ? 0 : all - whole;
      const int kept = all > 1 ? all : 0;
      int run = mine, run_all = kept;
#pragma unroll 1
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, run, d), up_all = __shfl_up_sync(0xffffffffu, run_all, d);
        if (lane >= d) run += up, run_all += up_all;
      }
      const unsigned past = __ballot_sync(0xffffffffu, base + run > id);
      if (past) {
        const int src = __ffs(past) - 1;
        r.n = n0 + src;
        r.len = __shfl_sync(0xffffffffu, len, src);
        r.count = __shfl_sync(0xffffffffu, all, src);
        r.s = turn != 1 ? r.count - 1 : id - __shfl_sync(0xffffffffu, base + run - mine, src);
        r.record = records + __shfl_sync(0xffffffffu, run_all - kept, src);
        r.t0 = seq_start(args, r.n);
      }
      base += __shfl_sync(0xffffffffu, run, 31);
      records += __shfl_sync(0xffffffffu, run_all, 31);
    }
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
// final states.  SIZED: FP16 keys as they are, K' times a power of two by the chunk's largest.
// (Unit keys' power is the same for all; asked for in each chunk it took 4% more.)
template <bool F16, bool LOCAL, bool SIZED>
__global__ void __launch_bounds__(kThreads, 1)
    lin_prefill_kernel(const LinPrefillArgs args, const __grid_constant__ LinMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + kBars);
  Scalars* scalars = reinterpret_cast<Scalars*>(smem + kScalars);
  // (by an exchange, so that the compiler knows it for the same in all lanes)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (LOCAL) grid_dependency_launch();
  const int HV = args.HV, h = blockIdx.x % HV, id = blockIdx.x / HV;
  const Segment seg = find_segment<LOCAL>(args, id, lane);
  if (!LOCAL && blockIdx.x == 0 && warp == kGateWarp)  // bounds of no sequence, which has no CTA of its own
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
  const int first = seg.s * seg.tokens;
  const bool last_segment = seg.s == seg.count - 1;
  const int L = last_segment ? seg.len - first : seg.tokens, nch = (L + kC - 1) / kC;
  const int64_t t0 = seg.t0 + first;
  if (LOCAL && last_segment) return;  // nothing starts from its state
  const int slot = args.state_idx[seg.n];
  if (tc::smem_u32(smem) & 1023u) {  // swizzled tiles start on 1024 bytes
    if (tid == 0) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
    leave();
    return;
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&bars.tmem, kTmCols);
  if (tid == 0) {
    bars.timed_out = 0;
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&bars.full[i], 1);
      tc::mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < kScalarBufs; ++i) {
      tc::mbar_init(&bars.gate_full[i], 1);
      tc::mbar_init(&bars.in_full[i], kNormWarps);
      tc::mbar_init(&bars.sc_free[i], kWorkers);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.wk_full[i], kWorkers);
      tc::mbar_init(&bars.ds_full[i], 1);
    }
    tc::mbar_init(&bars.u_full, kWorkers);
    tc::mbar_init(&bars.p_full, kWorkers);
    tc::mbar_init(&bars.qk_full, 1);
    tc::mbar_init(&bars.o_full, 1);
    tc::mbar_init(&bars.drained, 1);
    tc::mbar_init(&bars.state_full, 1);
    tc::mbar_init(&bars.state_read, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem, 0);
  if (slot < 0 || slot >= args.pool_slots) {  // padding or out of range: zero outputs, no state touched
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmCols);
    if (!LOCAL) {
      if (slot != -1 && tid == 0 && h == 0 && seg.s == 0) set_error(args.err_flag, KDA_DEVERR_SLOT);
      for (int64_t i = tid; i < (int64_t)L * 16; i += kThreads)
        *reinterpret_cast<uint4*>(args.o + ((t0 + i / 16) * HV + h) * kHeadDim + (i % 16) * 8) = make_uint4(0, 0, 0, 0);
    }
    leave();
    return;
  }
  const bool from_pool = seg.s == 0 && (LOCAL || seg.count == 1);
  const LinGateArgs& ga = args.gate;
  // FP16: unit keys are at most 1 and become K' times 2^15, so that small ones keep their places;
  // keys as they are times a power of two by the chunk's largest (K' made of them alone ended at
  // 2^-24: states 4e-5 of their RMS off for keys of size 1e-3)
  constexpr float k_up = F16 && !SIZED ? 32768.f : 1.f;
  bool ok = true;

  // 768 threads start with 80 registers each; 512 at 96 and 256 at 48 are those 61440
  if (warp < kWorkers) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    // A warp that runs out of time goes on without waiting and without arriving, so
    // that the others meet it at their barrier and run out too.
    const int quad = warp & 3, part = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    auto done = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0 && ok) arrive(bar);
    };

    auto await = [&](uint64_t* bar, uint32_t phase) { ok = ok && warp_wait(bar, phase); };
    constexpr int kStage = LOCAL ? kLocalStage : kStageBytes, kK = LOCAL ? 0 : kTile;

    // ------------------------------------------------------------------------- K'
    // 4 rows a warp; of its row a thread has a 16-byte piece of either half of the channels
    const int row = 4 * warp + (lane >> 3), x8 = lane & 7;
    auto key_power = [&](const Scalars& sc, float& back) {
      const float4 m = *reinterpret_cast<const float4*>(sc.k_big);  // (in order as whole numbers, NaN the largest)
      return to_2p15(max(max(__float_as_uint(m.x), __float_as_uint(m.y)), max(__float_as_uint(m.z), __float_as_uint(m.w))) >> 23, back);
    };
    auto keys = [&](int c, int st, const Scalars& sc) {
      await(&bars.in_full[c % kScalarBufs], c / kScalarBufs);
      const int left = L - c * kC;
      uint8_t* rows = smem + st * kStage + kK;
      uint8_t* to = smem + (LOCAL ? kStages * kLocalStage + (c & 1) * kLocalWk : kWk);
      const float wk = sc.w[row];
      uint4 kw[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) kw[p] = *line16(rows + p * 8192, row, x8);
      if (row >= left) {  // the next sequence's values and keys: NaN times zero is NaN
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          *line16(rows + kTile + p * 8192, row, x8) = make_uint4(0, 0, 0, 0);
          kw[p] = make_uint4(0, 0, 0, 0);
        }
      }
      float w = row < left ? wk : 0.f, back;
      if (SIZED) w *= key_power(sc, back);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t x[4] = {kw[p].x, kw[p].y, kw[p].z, kw[p].w};
        uint32_t piece[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 f = mul2(widen2<F16>(x[e]), make_float2(w, w)), rest;
          piece[0][e] = round2<F16>(f, rest);
          piece[1][e] = round2<F16>(rest, f);
          if (!F16) piece[2][e] = round2<F16>(f, rest);
        }
#pragma unroll
        for (int i = 0; i < (F16 ? 2 : 3); ++i)
          *line16(to + i * kTile + p * 8192, row, x8) = make_uint4(piece[i][0], piece[i][1], piece[i][2], piece[i][3]);
      }
    };

    // --------------------------------------------------------------------- state
    const int dv = 32 * quad + lane;  // this thread's value column; its key channels 32 part ..
    uint8_t* box = smem + (part == 3 ? kP : (LOCAL ? kLocalState : kState) + part * kTile);  // of the pool's state
    float S[32];
    auto record = [&](int64_t segment) { return args.local_state + (segment * HV + h) * 4096 + tid; };
    auto start = [&]() {
    // (The first launch leaves the pool as it is: what it does not leave behind can be
    // read while it runs, and a sequence in one piece needs nothing of it.)
    if (!LOCAL && seg.count > 1) grid_dependency_wait();
    if (from_pool) {
      await(&bars.state_full, 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(line16(box, dv, j));
        S[4 * j] = x.x, S[4 * j + 1] = x.y, S[4 * j + 2] = x.z, S[4 * j + 3] = x.w;
      }
      asm volatile("barrier.cta.sync 1, 512;" ::: "memory");  // its place is others' now
      if (!LOCAL && tid == 0 && ok) arrive(&bars.state_read);
    }
    if (seg.s == 0) {
      // The CTA of the last segment writes the sequence's slot, maybe before this one
      // reads it: the first launch leaves a copy where the last segment has no record.
      float4* copy = record(seg.record + seg.count - 1);
      if (LOCAL) {
#pragma unroll
        for (int j = 0; j < 8; ++j) copy[j * 512] = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
      } else if (seg.count > 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 x = __ldcg(copy + j * 512);
          S[4 * j] = x.x, S[4 * j + 1] = x.y, S[4 * j + 2] = x.z, S[4 * j + 3] = x.w;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) S[j] = 0.f;
    }
    if (!LOCAL && seg.s > 0) {
      // `up`: decay from the end of a segment before to the start of this one.  Where it is
      // zero, segments that are not finite still count (NaN), as they do in one piece.
      const float* d = args.local_decay + (int64_t)seg.record * HV + h;
      float up = 1.f;
      for (int m0 = seg.s - 1; m0 >= 0; m0 -= 32) {
        const float here = m0 >= lane ? __ldcg(d + (int64_t)(m0 - lane) * HV) : 0.f;
        const unsigned bad = __ballot_sync(0xffffffffu, __float_as_int(here) < 0);
        for (int i = 0; i < 32 && i <= m0; ++i) {
          if (up == 0.f) {
            if (bad >> i == 0) break;
            i += __ffs(bad >> i) - 1;
          }
          const float4* src = record(seg.record + m0 - i);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 x = __ldcg(src + j * 512);
            S[4 * j] = fmaf(up, x.x, S[4 * j]);
            S[4 * j + 1] = fmaf(up, x.y, S[4 * j + 1]);
            S[4 * j + 2] = fmaf(up, x.z, S[4 * j + 2]);
            S[4 * j + 3] = fmaf(up, x.w, S[4 * j + 3]);
          }
          up *= fabsf(__shfl_sync(0xffffffffu, here, i));
        }
      }
    }
    };
    float decay = 1.f, last = 1.f, k_down = 1.f / k_up;  // of the chunk whose dS is under way
    auto take = [&](const Scalars& sc) {
      last = sc.last;
      if (SIZED) key_power(sc, k_down);
    };
    auto update = [&](int c) {  // S of the next chunk
      tc::tc_fence_after();
      uint32_t r[2][16];
#pragma unroll
      for (int g = 0; g < 2; ++g)
        tc::tmem_ld16_async(lanes + kTmU + (LOCAL ? 128 * (c & 1) : 0) + 32 * part + 16 * g, r[g]);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        wait_ld(r[g]);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          float2 u = make_float2(__uint_as_float(r[g][j]), __uint_as_float(r[g][j + 1]));
          if (F16) u = mul2(u, make_float2(k_down, k_down));
          const float2 x = fma2(make_float2(last, last), make_float2(S[16 * g + j], S[16 * g + j + 1]), u);
          S[16 * g + j] = x.x;
          S[16 * g + j + 1] = x.y;
        }
      }
      decay *= last;
    };
    // S^T as an operand; FP16: a row times a power of two by its largest
    auto power = [&](int c) {
      float down = 1.f;
      if constexpr (F16) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) m = fmaxf(m, fabsf(S[j]));
        bars.s_big[c & 1][part][dv] = (uint8_t)(__float_as_uint(m) >> 23);
        asm volatile("barrier.cta.sync 1, 512;" ::: "memory");
        uint32_t x = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) x = max(x, (uint32_t)bars.s_big[c & 1][i][dv]);
        float back;
        down = to_2p15(x, back);
        if (part == 0) bars.s_scale[c % 3][dv] = back;
      }
      return down;
    };
    auto operand = [&](int half, float down) {  // (and wait_st)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float2 x = make_float2(S[16 * g + 2 * j], S[16 * g + 2 * j + 1]), rest;
          if (F16) x = mul2(x, make_float2(down, down));
          w[j] = round2<F16>(x, rest);
          if (half) w[j] = round2<F16>(rest, x);
        }
        tmem_st8(lanes + kTmS + 64 * half + 16 * part + 8 * g, w);
      }
    };

    // ------------------------------------------------------------------------- P
    // rows r0 and r0 + 8 of a 16 x 16 block, block `part` of the rows' four
    const int r0 = 16 * quad + (lane >> 2), turn = r0 & 7;
    uint8_t* at[2];  // where columns 2 (lane % 4) and + 1 of a row's first piece are, but for the swizzle
#pragma unroll
    for (int e = 0; e < 2; ++e) at[e] = smem + kP + (r0 + 8 * e) * 128 + 4 * (lane & 3);
    auto put = [&](int j, int e, uint32_t hi, uint32_t lo) {
      uint8_t* to = at[e] + ((j ^ turn) << 4);
      *reinterpret_cast<uint32_t*>(to) = hi;
      *reinterpret_cast<uint32_t*>(to + kTile / 2) = lo;
    };
    auto weights = [&](int c, const Scalars& sc, float s_down) {
      await(&bars.qk_full, c);
      tc::tc_fence_after();
      float2 down[2];  // FP16: powers of two of the rows
      if constexpr (F16) {  // |q.k| is at most |q| |k|
        float k2 = 1.f;
        if (!ga.use_qk_l2norm) {
          k2 = fmaxf(sc.kk[lane], sc.kk[lane + 32]);
          k2 = sqrtf(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(k2))));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float back;
          down[e].x = down[e].y = to_2p15(__float_as_uint(sc.big[r0 + 8 * e] * k2) >> 23, back);
          if (part == 0 && (lane & 3) == 0) bars.p_scale[c & 1][r0 + 8 * e] = back;
        }
      }
      if (part > quad) operand(1, s_down);
      if (part <= quad) {
        const uint32_t qk = lanes + kTmO + 64 * (c & 1) + 16 * part;
        uint32_t r[2][4];
        ld_frag8(qk, r[0]);
        ld_frag8(qk + 8, r[1]);
        const bool far = sc.far[quad] != 0;
        operand(1, s_down);  // (while these come)
        wait_ld(r[0]);
        wait_ld(r[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = 16 * part + 8 * i + 2 * (lane & 3);
          float2 x[2];
          if (!far) {
            const float2 f = *reinterpret_cast<const float2*>(&sc.col[quad][col]);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              x[e] = mul2(f, make_float2(__uint_as_float(r[i][2 * e]), __uint_as_float(r[i][2 * e + 1])));
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 c_i = make_float2(sc.c_hi[r0 + 8 * e], sc.c_lo[r0 + 8 * e]);
              x[e].x = sc.k[col] * exp_diff(c_i, make_float2(sc.c_hi[col], sc.c_lo[col])) * __uint_as_float(r[i][2 * e]);
              x[e].y = sc.k[col + 1] * exp_diff(c_i, make_float2(sc.c_hi[col + 1], sc.c_lo[col + 1])) *
                       __uint_as_float(r[i][2 * e + 1]);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (F16) x[e] = mul2(x[e], down[e]);
            if (part == quad) {
              const int i_row = r0 + 8 * e;
              x[e].x = col <= i_row ? x[e].x : 0.f;
              x[e].y = col < i_row ? x[e].y : 0.f;
            }
            float2 rest;
            const uint32_t hi = round2<F16>(x[e], rest), lo = round2<F16>(rest, x[e]);
            put(2 * part + i, e, hi, lo);
          }
        }
      }
      wait_st();
      tc::tc_fence_before();
      done(&bars.p_full);
    };

    // ------------------------------------------------------------------- outputs
    // 32 value columns a warp, 16 tokens a thread
    const int odd = lane & 1;
    const uint32_t pick = odd ? 0x3276u : 0x5410u;
    const int64_t step = (int64_t)HV * kHeadDim;
    kda_bf16* dst = args.o + ((t0 + 16 * part + odd) * HV + h) * kHeadDim + ((32 * quad + lane) & ~1);
    // (their products have been waited for, before the next chunk's operand)
    auto outputs = [&](int c, const Scalars& sc, uint64_t* free) {
      const int tok = 16 * part, left = L - c * kC - tok - odd;
      tc::tc_fence_after();
      const float up = F16 ? bars.s_scale[c % 3][dv] : 1.f;
      uint32_t y2[8];  // two tokens of one column each
      uint32_t q[16], r[16];
      tc::tmem_ld16_async(lanes + kTmQ + 64 * (c & 1) + tok, q);
      tc::tmem_ld16_async(lanes + kTmO + 64 * (c & 1) + tok, r);
      wait_ld(q);
      wait_ld(r);
      {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t2 = tok + 2 * j;
          float2 f = *reinterpret_cast<const float2*>(sc.out + t2), rest;
          float2 y = mul2(*reinterpret_cast<const float2*>(sc.row + t2),
                          make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])));
          if (F16) {
            f = mul2(f, make_float2(up, up));
            y = mul2(y, *reinterpret_cast<const float2*>(bars.p_scale[c & 1] + t2));
          }
          y2[j] = round2<F16>(fma2(f, make_float2(__uint_as_float(q[2 * j]), __uint_as_float(q[2 * j + 1])), y), rest);
        }
      }
      tc::tc_fence_before();
      done(free);
#pragma unroll
      for (int j = 0; j < 8; ++j)  // traded for two columns of one token each
        y2[j] = __byte_perm(y2[j], __shfl_xor_sync(0xffffffffu, y2[j], 1), pick);
      if (c < nch - 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) *reinterpret_cast<uint32_t*>(dst + 2 * j * step) = y2[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (2 * j < left) *reinterpret_cast<uint32_t*>(dst + 2 * j * step) = y2[j];
      }
      dst += kC * step;
    };

    auto stage = [&](int c) { return c % kStages; };
    auto factors = [&](int c) -> Scalars& { return scalars[c % kScalarBufs]; };
    keys(0, stage(0), factors(0));
    done(&bars.wk_full[0]);
    start();  // (the first launch may still be running)
    if (!LOCAL && part > quad)  // right of the diagonal all is zero, and stays so
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) put(2 * part + i, e, 0, 0);
    if (LOCAL) {
      // K' and dS are there twice: a chunk's product runs while the next one's K' is made
      for (int c = 0; c < nch; ++c) {
        if (c > 0) {
          await(&bars.ds_full[(c - 1) & 1], (c - 1) >> 1);
          update(c - 1);
        }
        take(factors(c));
        if (c + 1 < nch) keys(c + 1, stage(c + 1), factors(c + 1));
        tc::tc_fence_before();
        if (c + 1 < nch) done(&bars.wk_full[(c + 1) & 1]);
        done(&bars.sc_free[c % kScalarBufs]);
      }
    } else {
      for (int c = 0; c < nch; ++c) {
        if (c > 0) update(c - 1);
        tc::tc_fence_before();
        done(&bars.u_full);
        take(factors(c));
        const float down = power(c);
        if (c > 0) {  // the last operand and the last P have been read
          await(&bars.o_full, c - 1);
          tc::tc_fence_after();
        }
        operand(0, down);
        weights(c, factors(c), down);
        if (c > 0) outputs(c - 1, factors(c - 1), &bars.sc_free[(c - 1) % kScalarBufs]);
        await(&bars.ds_full[c & 1], c >> 1);  // K' has been read, dS is there
        if (c + 1 < nch) {
          keys(c + 1, stage(c + 1), factors(c + 1));
          done(&bars.wk_full[(c + 1) & 1]);
        }
      }
      await(&bars.o_full, nch - 1);
      outputs(nch - 1, factors(nch - 1), &bars.sc_free[(nch - 1) % kScalarBufs]);
    }
    if (LOCAL) await(&bars.ds_full[(nch - 1) & 1], (nch - 1) >> 1);
    if (LOCAL || last_segment) {
      update(nch - 1);
      if (LOCAL) {
        float4* to = record(seg.record + seg.s);
#pragma unroll
        for (int j = 0; j < 8; ++j) to[j * 512] = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
        float zero = 0.f;  // NaN where one is not finite
#pragma unroll
        for (int j = 0; j < 32; ++j) zero = fmaf(S[j], 0.f, zero);
        if (any_worker(zero != 0.f)) decay = -decay;
        if (tid == 0) args.local_decay[(int64_t)(seg.record + seg.s) * HV + h] = decay;
      } else {  // back to the pool as it came; all products are done
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(line16(box, dv, j)) = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
        if (!ok) bars.timed_out = 1;
        tc::fence_async_smem();
        asm volatile("barrier.cta.sync 1, 512;" ::: "memory");
        if (tid == 0 && !*static_cast<volatile int*>(&bars.timed_out)) {
#pragma unroll
          for (int a = 0; a < 4; ++a)
            tma_store_box(&maps.pool, a * 32, 0, (slot * HV + h) * kHeadDim, smem + (a == 3 ? kP : kState + a * kTile));
          tc::bulk_commit();
          tc::bulk_wait_read();  // shared memory stays until then
        }
      }
    }
  } else {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
  if (warp == kRowWarp) {
    // ------------------------------------------------------------------------ rows
    constexpr int kStage = LOCAL ? kLocalStage : kStageBytes;
    const bool leader = elect_one();
    int issued = 0;
    for (int c = 0; c < nch; ++c) {
      const int st = c % kStages;
      if (c >= kStages && !(ok = warp_wait(&bars.empty[st], c / kStages - 1))) break;
      if (!LOCAL && c == 2 && from_pool && !(ok = warp_wait(&bars.state_read, 0))) break;
      uint8_t* rows = smem + st * kStage;
      if (leader) {
        uint64_t* bar = &bars.full[st];
        tc::mbar_expect_tx(bar, kStage);
        const int tok = (int)t0 + c * kC;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          if (!LOCAL) tma_box(rows + a * 8192, &maps.q, a * 64, h / args.G, tok, bar);
          tma_box(rows + kStage - 2 * kTile + a * 8192, &maps.k, a * 64, h / args.G, tok, bar);
          tma_box(rows + kStage - kTile + a * 8192, &maps.v, a * 64, h, tok, bar);
        }
        if (c == 0 && from_pool) {
          tc::mbar_expect_tx(&bars.state_full, 4 * kTile);
          uint8_t* to = smem + (LOCAL ? kLocalState : kState);
#pragma unroll
          for (int a = 0; a < 4; ++a)
            tma_box(a == 3 ? smem + kP : to + a * kTile, &maps.pool, a * 32, 0, (slot * HV + h) * kHeadDim, &bars.state_full);
        }
      }
      __syncwarp();
      issued = c + 1;
    }
    // nothing may land after the CTA is gone
    for (int c = issued > kStages ? issued - kStages : 0; c < issued; ++c) warp_wait(&bars.full[c % kStages], c / kStages);
    if (from_pool) warp_wait(&bars.state_full, 0);
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------------------- products
    constexpr uint32_t kType = F16 ? tc::idesc_f16_f32(128, 64) : tc::idesc_bf16_f32(128, 64);
    constexpr uint32_t kIdU = (F16 ? tc::idesc_f16_f32(128, 128) : tc::idesc_bf16_f32(128, 128)) | tc::kIdescMnA | tc::kIdescMnB;
    constexpr uint32_t kIdP = F16 ? tc::idesc_f16_f32(64, 64) : tc::idesc_bf16_f32(64, 64);
    const bool leader = elect_one();
    if (LOCAL) {
      for (int c = 0; c < nch; ++c) {
        const uint64_t v_op = tc::sw128_desc_mn(tc::smem_u32(smem + c % kStages * kLocalStage) + kTile, 8192);
        const uint64_t wk_op = tc::sw128_desc_mn(tc::smem_u32(smem + kStages * kLocalStage) + (c & 1) * kLocalWk, 8192);
        // K' of chunk c, behind the state's update by dS of c - 2
        if (!(ok = warp_wait(&bars.in_full[c % kScalarBufs], c / kScalarBufs) && warp_wait(&bars.wk_full[c & 1], c >> 1))) break;
        tc::fence_async_smem();
        tc::tc_fence_after();
        if (leader) {  // dS^T = V^T K'
#pragma unroll
          for (int b = 0; b < (F16 ? 2 : 3); ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tc::mma_bf16(tmem + kTmU + 128 * (c & 1), v_op + ((j * 2048) >> 4), wk_op + ((b * kTile + j * 2048) >> 4), kIdU,
                           b + j > 0);
          tc::mma_commit(&bars.ds_full[c & 1]);
          tc::mma_commit(&bars.empty[c % kStages]);
        }
        __syncwarp();
      }
    } else {
      const uint64_t wk_op = tc::sw128_desc_mn(tc::smem_u32(smem + kWk), 8192), p_op = tc::sw128_desc(tc::smem_u32(smem + kP));
      for (int c = 0; c < nch; ++c) {
        const int st = c % kStages;
        const uint32_t rows = tc::smem_u32(smem + st * kStageBytes), turn = 64 * (c & 1);
        const uint64_t q_op = tc::sw128_desc(rows), k_op = tc::sw128_desc(rows + kTile);
        const uint64_t v_op = tc::sw128_desc_mn(rows + 2 * kTile, 8192);
        // K' is the last of what a chunk needs before its state; the outputs of c - 2,
        // whose place Q K^T takes, were read before
        if (!(ok = warp_wait(&bars.in_full[c % kScalarBufs], c / kScalarBufs) && warp_wait(&bars.wk_full[c & 1], c >> 1))) break;
        tc::fence_async_smem();
        tc::tc_fence_after();
        if (leader) {  // Q K^T
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint64_t off = ((j >> 2) * 8192 + (j & 3) * 32) >> 4;
            tc::mma_bf16(tmem + kTmO + turn, q_op + off, k_op + off, kIdP, j > 0);
          }
          tc::mma_commit(&bars.qk_full);
        }
        __syncwarp();
        if (!(ok = warp_wait(&bars.u_full, c))) break;
        tc::tc_fence_after();
        if (leader) {
#pragma unroll
          for (int b = 0; b < (F16 ? 2 : 3); ++b)  // dS^T = V^T K'
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tc::mma_bf16(tmem + kTmU, v_op + ((j * 2048) >> 4), wk_op + ((b * kTile + j * 2048) >> 4), kIdU, b + j > 0);
          tc::mma_commit(&bars.ds_full[c & 1]);
        }
        __syncwarp();
        if (!(ok = warp_wait(&bars.p_full, c))) break;
        tc::fence_async_smem();
        tc::tc_fence_after();
        if (leader) {  // O1^T = S^T Q^T, O2^T = V^T P^T
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              mma_ts(tmem + kTmQ + turn, tmem + kTmS + 64 * b + 8 * j, q_op + (((j >> 2) * 8192 + (j & 3) * 32) >> 4), kType,
                     b + j > 0);
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tc::mma_bf16(tmem + kTmO + turn, v_op + ((j * 2048) >> 4), p_op + ((b * (kTile / 2) + j * 32) >> 4),
                           kType | tc::kIdescMnA, b + j > 0);
          tc::mma_commit(&bars.empty[st]);
          tc::mma_commit(&bars.o_full);
        }
        __syncwarp();
      }
    }
  } else if (warp < kNormWarp) {
    // ----------------------------------------------------------- the decays' factors
    // one of two warps, every other chunk
    const float log_rate = ga.A_log ? ga.A_log[h] : 0.f, bias = ga.dt_bias ? ga.dt_bias[h] : 0.f;
    ushort2 next[2];  // of tokens 2 lane and 2 lane + 1
    auto load_gate = [&](int c) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        next[e] = make_ushort2(0, 0);
        if (c * kC + 2 * lane + e < L) next[e] = lin_gate_load(ga, (t0 + c * kC + 2 * lane + e) * HV + h);
      }
    };
    load_gate(warp - kGateWarp);
    const float neg_rate = ga.A_log ? -expf(log_rate) : 0.f;
#pragma unroll 1
    for (int c = warp - kGateWarp; c < nch; c += 2) {
      const int left = L - c * kC, sb = c % kScalarBufs;
      Scalars& sc = scalars[sb];
      float g[2];
#pragma unroll 1
      for (int e = 0; e < 2; ++e) g[e] = 2 * lane + e < left ? lin_log_decay<F16>(ga, e ? next[1] : next[0], neg_rate, bias) : 0.f;
      load_gate(c + 2);
      float2 run = pair_add(make_float2(g[0], 0.f), make_float2(g[1], 0.f));  // c of token 2 lane + 1
#pragma unroll 1
      for (int d = 1; d < 32; d <<= 1) {
        const float2 up = make_float2(__shfl_up_sync(0xffffffffu, run.x, d), __shfl_up_sync(0xffffffffu, run.y, d));
        if (lane >= d) run = pair_add(up, run);
      }
      const float2 even = pair_add(run, make_float2(-g[1], 0.f));  // of token 2 lane
      if (c >= kScalarBufs && !(ok = warp_wait(&bars.sc_free[sb], c / kScalarBufs - 1))) break;
      auto put2 = [&](float* to, float a, float b) { *reinterpret_cast<float2*>(to + 2 * lane) = make_float2(a, b); };
      const float2 c_last = pair_from(run, 31);
      put2(sc.w, 2 * lane < left ? k_up * exp_diff(c_last, even) : 0.f, 2 * lane + 1 < left ? k_up * exp_diff(c_last, run) : 0.f);
      if (lane == 31) sc.last = expf(run.x + run.y);
      if (!LOCAL) {
        put2(sc.c_hi, even.x, run.x);
        put2(sc.c_lo, even.y, run.y);
        put2(sc.k, 1.f, 1.f);
        put2(sc.out, ga.scale * expf(even.x + even.y), ga.scale * expf(run.x + run.y));
        const float2 start = pair_from(even, lane & 24), end = pair_from(run, lane | 7);
        const bool far = !((start.x - end.x) + (start.y - end.y) <= kFar);
        const float2 c_b = make_float2(0.5f * (start.x + end.x), 0.f);
        if ((lane & 7) == 0) sc.far[lane >> 3] = far;
        const float e0 = far ? 1.f : exp_diff(even, c_b), e1 = far ? 1.f : exp_diff(run, c_b);
        put2(sc.row, ga.scale * e0, ga.scale * e1);
        if (F16) put2(sc.big, 1.f / e0, 1.f / e1);
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          const float2 ref = make_float2(__shfl_sync(0xffffffffu, c_b.x, 8 * x), 0.f);
          const bool some = lane < 8 * x + 8;
          put2(sc.col[x], some ? exp_diff(ref, even) : 0.f, some ? exp_diff(ref, run) : 0.f);
        }
      }
      __syncwarp();
      if (lane == 0) arrive(&bars.gate_full[sb]);
    }
  } else {
    // ------------------------------------------------------------------------ norms
    // The squares of 16 rows are the diagonal of the rows times themselves, by
    // register-to-register products: of K, then of Q.
    const int r16 = 16 * (warp - kNormWarp) + (lane & 15);
    const bool l2 = ga.use_qk_l2norm, upper = lane >= 16;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      Scalars& sc = scalars[c % kScalarBufs];
      if (!(ok = warp_wait(&bars.full[c % kStages], c / kStages))) break;
      float n[2];
      if (l2 || F16) {
        const uint32_t tile = tc::smem_u32(smem + c % kStages * (LOCAL ? kLocalStage : kStageBytes));
#pragma unroll 1
        for (int b = 0; b < (LOCAL ? 1 : 2); ++b) {
          const uint32_t at = tile + (b == 0 && !LOCAL ? kTile : 0) + r16 * 128;
          float lo[2][4] = {}, hi[2][4] = {};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t f[4];
            ldm4(at + (k >> 2) * 8192 + ((((k & 3) * 2 + (lane >> 4)) ^ (r16 & 7)) << 4), f);
            mma16<F16>(lo[k & 1], f, f[0], f[2]);
            mma16<F16>(hi[k & 1], f, f[1], f[3]);
          }
          // row g of lo is in lane 4 g + g / 2, and so is row g + 8 of hi
          const int odd = lane >> 2 & 1, from = 4 * (lane & 7) + ((lane & 7) >> 1);
          const float d_lo = __shfl_sync(0xffffffffu, odd ? lo[0][1] + lo[1][1] : lo[0][0] + lo[1][0], from);
          const float d_hi = __shfl_sync(0xffffffffu, odd ? hi[0][3] + hi[1][3] : hi[0][2] + hi[1][2], from);
          (b ? n[1] : n[0]) = lane & 8 ? d_hi : d_lo;
        }
      }
      if (!(ok = warp_wait(&bars.gate_full[c % kScalarBufs], c / kScalarBufs))) break;
      if (l2) {
        const float rk = rsqrtf(n[0] + kNormEps);
        if (upper) sc.w[r16] *= rk;
        if (!LOCAL) {
          if (!upper) sc.k[r16] = rk;
          sc.col[upper ? 1 : 0][r16] *= rk;
          sc.col[upper ? 3 : 2][r16] *= rk;
          (upper ? sc.row : sc.out)[r16] *= rsqrtf(n[1] + kNormEps);
        }
      }
      // |k_j|^2 of this sequence's keys, one that is not finite for FP16's largest: the others keep
      // their places
      const float k2 = r16 >= L - c * kC ? 0.f : n[0] < 5.5e11f ? n[0] : 5.5e11f;
      if (SIZED) {
        const float m = sc.w[r16] * sqrtf(k2);
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if (lane == 0) sc.k_big[warp - kNormWarp] = __uint_as_float(most);
      }
      if (F16 && !LOCAL) {
        if (upper) sc.big[r16] *= sqrtf(n[1]);
        else sc.kk[r16] = k2;
      }
      __syncwarp();
      if (lane == 0) arrive(&bars.in_full[c % kScalarBufs]);
    }
  }
  }
  // All products have been waited for but those whose results nobody needs; where a
  // wait has run out, with a limit, before TMEM and shared memory go.
  if (!ok) bars.timed_out = 1;
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == kMmaWarp) {
    if (elect_one()) tc::mma_commit(&bars.drained);  // the same lane as issued them
    __syncwarp();
    warp_wait(&bars.drained, 0);
  }
  if (bars.timed_out && tid == 0) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
  leave();
  __syncthreads();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmCols);
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

// The same of a pool of FP32 states, box (32 key channels, 1, 128 value columns).
bool encode_pool(CUtensorMap* m, const void* base, int64_t rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)kHeadDim, 1u, (cuuint64_t)rows};
  const cuuint64_t stride[2] = {(cuuint64_t)kHeadDim * 4, (cuuint64_t)kHeadDim * 4};
  const cuuint32_t box[3] = {32u, 1u, (cuuint32_t)kHeadDim};
  const cuuint32_t estride[3] = {1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dim, stride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using Kernel = void (*)(LinPrefillArgs, LinMaps);
Kernel pick(bool f16, bool sized, bool local) {
  if (!f16) return local ? lin_prefill_kernel<false, true, false> : lin_prefill_kernel<false, false, false>;
  if (!sized) return local ? lin_prefill_kernel<true, true, false> : lin_prefill_kernel<true, false, false>;
  return local ? lin_prefill_kernel<true, true, true> : lin_prefill_kernel<true, false, true>;
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
  for (bool local : {false, true})
    for (const Kernel kernel : {pick(false, false, local), pick(true, false, local), pick(true, true, local)})
      if (!allow(kernel)) return KDA_ERR_CUDA;
  ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  return KDA_OK;
}

// Tokens of a segment.  Sequences of one length: the number of segments each that
// takes least, by what a chunk and a CTA's start cost in thousands of cycles (measured:
// 4.7 and 6 in the second launch, 2.3 and 5 in the first, which the last segments are
// spared).  With lengths that differ much (one of more than 1.25 times the mean), segments
// of an SM's share of the chunks, at least 4, for sequences of more than 1.6 of them; of
// half a share, for sequences of more than 1.5 shares, where that is 16 chunks or more;
// and below 2 for all.  In a model of the SMs with these costs that takes 1 to 7% longer
// than the best lengths for each of 500 batches, half shares throughout 11 to 20%.
struct Segments {
  int even, ragged, even_most, uncut;
  int64_t most, whole, records;  // segments, whole segments, segments of sequences in several: at most
};
Segments cut(const kda_dims& d, int num_seqs, int64_t total_tokens, int64_t sms) {
  Segments r{};
  const int64_t len = (total_tokens + num_seqs - 1) / num_seqs, chunks = (len + kC - 1) / kC, heads = (int64_t)num_seqs * d.HV;
  double best = 1e300;
  int64_t even = chunks;
  for (int64_t n = 1; n <= chunks && n <= 64; ++n) {
    const int64_t each = (chunks + n - 1) / n, got = (chunks + each - 1) / each;
    const int64_t waves = (heads * got + sms - 1) / sms, waves1 = (heads * (got - 1) + sms - 1) / sms;
    const double cost = waves * (4.7 * each + 6) + waves1 * (2.3 * each + 5);
    if (cost < best) best = cost, even = each;
  }
  const int64_t share = (total_tokens * d.HV / sms + kC - 1) / kC, few = share < 16 ? share : (share + 1) / 2;
  const int64_t even_most = len + len / 4, ragged = (few < 4 ? 4 : few) * kC;
  const int64_t uncut = share <= 2 ? ragged : share < 16 ? ragged * 8 / 5 : ragged * 3;
  const bool pieces = even < chunks, may_differ = num_seqs > 1 && total_tokens > uncut;
  const int64_t L = pieces || num_seqs == 1 ? even * kC : (even_most + kC - 1) / kC * kC;
  auto tokens = [](int64_t n) { return (int)(n < INT32_MAX ? n : INT32_MAX / kC * kC); };
  r.even = tokens(L);
  r.ragged = tokens(ragged);
  r.uncut = tokens(uncut);
  r.even_most = num_seqs == 1 ? INT32_MAX : tokens(even_most);
  r.most = num_seqs;
  auto count = [&](int64_t n) {
    const int64_t whole = total_tokens / n, records = whole < num_seqs ? 2 * whole : whole + num_seqs;
    r.most = whole + num_seqs > r.most ? whole + num_seqs : r.most;
    r.whole = whole > r.whole ? whole : r.whole;
    r.records = records > r.records ? records : r.records;
  };
  if (pieces) count(L);
  if (may_differ) count(ragged);
  return r;
}
// The workspace size does not depend on the device: so many SMs as this GPU has.
constexpr int64_t kSms = 152;

}  // namespace
}  // namespace kda

using namespace kda;

// A record of what each segment adds, and its decay; none where no sequence can
// have two segments.
extern "C" size_t kda_lin_prefill_workspace_size(kda_dims dims, int num_seqs, int64_t total_tokens) {
  if (num_seqs < 0 || total_tokens < 0 || dims.H <= 0 || dims.HV <= 0) return 0;
  if (total_tokens > INT32_MAX) return SIZE_MAX;  // refused; no capacity check may pass
  if (num_seqs == 0 || total_tokens == 0) return 0;
  return (size_t)cut(dims, num_seqs, total_tokens, kSms).records * dims.HV * (65536 + 16);
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
  args.pool_slots = pool_slots;
  args.state_idx = state_idx;
  args.cu_seqlens = cu_seqlens;
  args.num_seqs = num_seqs;
  args.total_tokens = total_tokens;
  args.each = total_tokens / num_seqs;
  args.o = o;
  const Segments c = cut(dims, num_seqs, total_tokens, kSms);
  args.seg_even = c.even;
  args.seg_ragged = c.ragged;
  args.even_most = c.even_most;
  args.uncut = c.uncut;
  args.err_flag = err_flag;
  const int64_t units = c.most * dims.HV, whole = c.whole * dims.HV;
  if (units > INT32_MAX) return KDA_ERR_SHAPE;
  args.local_state = static_cast<float4*>(workspace);
  args.local_decay = reinterpret_cast<float*>(static_cast<char*>(workspace) + (need > 0 ? (size_t)c.records * dims.HV * 65536 : 0));
  LinMaps m;
  if (!encode_rows(&m.q, q, dims.H, total_tokens) || !encode_rows(&m.k, k, dims.H, total_tokens) ||
      !encode_rows(&m.v, v, dims.HV, total_tokens) ||
      !encode_pool(&m.pool, state_pool, (pool_slots > 0 ? (int64_t)pool_slots : 1) * dims.HV * kHeadDim))
    return KDA_ERR_CUDA;
  s = allow_all();
  if (s != KDA_OK) return s;
  const bool f16 = dims.dtype == KDA_DTYPE_F16, sized = f16 && !gate.use_qk_l2norm;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  record_stage(0, st);
  // (without cu_seqlens the lengths are known here)
  const bool local = need > 0 && (cu_seqlens || args.each > c.even);
  if (local) {
    s = launch_dependent(pick(f16, sized, true), (unsigned)whole, kThreads, kSmem, false, st, args, m);
    if (s != KDA_OK) return s;
  }
  record_stage(1, st);
  s = launch_dependent(pick(f16, sized, false), (unsigned)units, kThreads, kSmem, local && !stage_between(), st, args, m);
  record_stage(2, st);
  return s;
}
