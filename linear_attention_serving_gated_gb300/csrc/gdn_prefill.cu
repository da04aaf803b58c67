// gdn_prefill.cu -- chunked varlen prefill of the gated delta rule with one
// decay per value head, on tcgen05/TMEM.
//
// Per (sequence, value head), 64 tokens at a time.  c_i is the log-decay summed
// up to token i of the chunk, r_i the inverse norm of its key, S (K x V) the
// state before the chunk:
//   A_ij = r_i r_j e^(c_i - c_j) k_i.k_j  (j < i),   T = (Diag(1 / beta) + A)^-1
//   X = K S,  Y_i = v_i - r_i e^(c_i) X_i,           D = T Y
//   O_i = scale rq_i e^(c_i) (Q S)_i + sum_(j <= i) P_ij D_j,
//         P_ij = scale rq_i r_j e^(c_i - c_j) q_i.k_j
//   S <- e^(c_last) S + sum_j e^(c_last - c_j) r_j k_j D_j^T
// One decay per head means that decays and norms only ever scale rows and
// columns of products, so the raw 16-bit q and k go into the tensor cores as
// they are: K K^T and Q K^T are exact up to FP32 sums, every exponent is of a
// difference c_i - c_j <= 0, and no decay is too strong for the chunk form.
//
// Two kernels.  Everything of a chunk that does not depend on the state is ready
// for all chunks at once:
//   gdn_chunk_kernel, a CTA of 128 threads per (chunk, value head), 4 per SM:
//     norms, decays, [K; Q] K^T on the tensor cores, A and P, T by blocks, and
//     one record of 33 KB (T, P, the chunk's row factors) for the second kernel.
// What is left is a chain of three dependent products a chunk.  Its latency, not
// bytes or flops, bounds a long sequence, so nothing else is on it.  16 chain
// warps hold the state in FP32 registers for the whole sequence and turn each
// product's TMEM accumulator into the next one's operand; one warp issues the
// products from behind hardware barriers, one Q S and P D, which only the output
// needs and 4 warps of their own join; two load the chunks' rows and records.
// Two forms of a CTA of that kernel, gdn_state_kernel:
//   narrow, a CTA per (sequence, value head, 32 value columns):
//       X  = K S           64 x 32 x 128
//       D  = T Y           64 x 32 x 64
//       dS = K^T D'       128 x 32 x 64, D'_j = e^(c_last - c_j) r_j D_j
//     S, Y and D' are right operands in shared memory, MN-major, the hi and lo
//     halves beside each other in one 64-wide tile: one product each for both.
//     M = 64 spreads the token rows over all four warp quadrants of TMEM, 16
//     lanes each, read in the fragment layout so that all 32 threads work.
//     thin, thinnest: the same with 16 and 8 value columns, 8 and 4 chain warps.
//   wide, a CTA per (sequence, value head), transposed:
//       X^T  = S^T K^T     128 x 64 x 128
//       D^T  = Y^T T^T     128 x 64 x 64
//       dS^T = D'^T K      128 x 128 x 64
//     Every product has the value columns as its rows, and what one's epilogue
//     makes is the next one's left operand, taken from TMEM: a thread's lane of
//     the accumulator becomes its lane of the operand, and nothing of the chain
//     passes through shared memory.
// A chunk takes 1.5 us in the narrow form, 1.2 in the thin one, 1.0 in the
// thinnest and 2.8 in the wide one, which does four times as many columns as the
// first: sequences that the SMs would wait for are as thin as they leave room
// for, the rest are wide (launch_states, pick_unit).
// Measured (whole call, in a graph): 1 x 4096 tokens, 16 heads, 96 us (8 heads
// 79), of which 18 pass before the chain starts; 8 x 4096 313; 16980 tokens in 8
// sequences with one of 8087 255; 1 x 128, 4 heads 11.  The chunk kernel alone: 23,
// 132 and 76 us of the first three.
// Precision: the state is FP32, in registers and in the pool.  As operands, S, T, Y
// and D' (and A in the inverse) are split in two BF16 halves, hi + lo, which leaves
// 2^-18; the products of two lo halves, 2^-18 again, are left out in the inverse and
// in the wide form.  States come out 4.6e-6 of their RMS off (an FP32 loop 1.6e-7),
// for keys that share nine tenths of a direction with beta near 1 up to 2.1e-5, the
// largest element 2.4e-4 of the RMS; the framework's bound for FP32 states is 1e-3,
// and outputs are rounded to 2^-9 or 2^-12.  A third half of T, Y and D' would take
// the wide form to 544 of TMEM's 512 columns and the FP16 form to 251 of 227 KB of
// shared memory.  P and D are split for the output: Q S and P D cancel where the
// state repeats what it is written, so that one rounding of P to BF16 showed up as 2
// per cent of the outputs' RMS.  K and Q are BF16 already.  FP16 K and Q are taken as they are for [K; Q] K^T; beside S
// and D', whose range is not FP16's, they are split exactly (11 bits into 8 + 8)
// by a pass over them that runs beside the chunk kernel.
#include <atomic>

#include "kda_host.h"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kC = 64;  // tokens per chunk
constexpr int kLdG = 20;  // row stride of the FP32 diagonal blocks of A

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
  uint8_t* records;    // one per (chunk, value head)
  int64_t max_chunks;  // ids the workspace holds
  int longest_first;   // the state kernel takes the sequences by length
  int most_narrow;     // at most so many sequences in the narrow form beside wide ones,
  int all_narrow;      // and whether all may take it
  int sms;
  int32_t* err_flag;
};

struct GdnMaps {
  CUtensorMap q, k, q_lo, k_lo;
};

// What the state kernels read of a chunk beside T and P.
struct ChunkScalars {
  float a[kC];  // -r_i e^(c_i)
  float s[kC];  // r_j e^(c_last - c_j), 0 past the sequence's end
  float o[kC];  // scale rq_i e^(c_i)
  float last;   // e^(c_last)
  float done;   // 1: the record is complete
  float pad[2];
};
// A chunk's record: T hi, T lo, P hi, P lo (tiles of 64 128-byte swizzled lines),
// scalars.
constexpr int kRecT = 0, kRecTlo = 8192, kRecP = 16384, kRecPlo = 24576, kRecScalars = 32768, kRecBytes = 33792;
static_assert(kRecScalars + sizeof(ChunkScalars) <= kRecBytes, "record");

// Shared memory of the chunk kernel: [K; Q] as two halves of 64 channels and
// 128 lines each and the scalars; P goes straight to the record.  A's hi and lo
// halves take the place of K, and T's that of Q, once their products are done.
struct ChunkCfg {
  static constexpr int kRowBytes = 32768;
  static constexpr int kScalars = kRowBytes;  // 1024 bytes
  static constexpr int kGate = kScalars + 1024;  // float hi[64], lo[64], beta[64], rk[64]
  static constexpr int kBar = kGate + 4 * kC * 4;
  static constexpr int kDiag = kBar + 64;  // A's diagonal blocks in FP32
  static constexpr int kSmem = kDiag + 4 * 16 * kLdG * 4;
  static constexpr int kTmCols = 64;
  // per SM; five of 96 registers take 500 instead of 507 us for 8 x 4096 tokens,
  // but 133 instead of 115 for 1 x 4096 (16 heads, whole call)
  static constexpr int kCtas = 4;
};

struct Bars {
  uint64_t key[3], key_free[3];  // rows of K and Q: landed (keys past the end zeroed: tail), consumed
  uint64_t tail;
  uint64_t rec[3], rec_free[3];  // records
  uint64_t x_full, xq_full, d_full, u_full;
  uint64_t o_full, o_read;
  uint64_t drained[2];  // all products of an issuing warp; used where a wait has run out
  int64_t chunk0;  // id of the sequence's first chunk
  uint32_t tmem;
  int timed_out;
};

// Roles of a state CTA's warps.
constexpr int kChainWarps = 16, kOutWarps = 4;
constexpr int kMmaWarp = kChainWarps + kOutWarps, kSideWarp = kMmaWarp + 1, kKeyWarp = kMmaWarp + 2,
              kRecWarp = kMmaWarp + 3, kStateThreads = (kRecWarp + 1) * 32;

// Forms of the state kernel.
enum { kThinnest, kThin, kNarrow, kWide, kMixed };
constexpr int kMaxSorted = 128;  // sequences a CTA ranks by length: two hundred cycles for 8, two thousand for 128

template <bool F16>
struct Cfg {
  static constexpr int kQ = 16384 * (F16 ? 2 : 1);  // K and Q; each before its low halves if FP16
  static constexpr int kKeyBytes = 2 * kQ;
  static constexpr int kKeys = F16 ? 2 : 3, kRecs = 2;     // chunks in shared memory: rows, records
  static constexpr int kRec = kKeys * kKeyBytes;
  static constexpr int kBars = kRec + kRecs * kRecBytes;
  // the narrow form's operands
  static constexpr int kS = (kBars + (int)sizeof(Bars) + 1023) / 1024 * 1024;
  static constexpr int kY = kS + 16384;
  static constexpr int kD = kY + 8192;
  static constexpr int kSmem = kD + 8192, kWideSmem = kBars + (int)sizeof(Bars);
};

// TMEM columns of the wide form.  Left operands (two BF16 a column): S, Y and
// after it D'.  Accumulators: X and after it D, dS, Q S, P D; a warp's quarter of
// D makes room for its D as an operand, 8 columns hi and 8 lo.  The narrow form
// has accumulators alone, in the same columns.
constexpr int kTmS = 0, kTmSlo = 64, kTmY = 128, kTmYlo = 160, kTmX = 192, kTmU = 256, kTmQ = 384, kTmO = 448,
              kTmCols = 512;

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
// The chain warps' wait: skipped once one has run out of time.
__device__ __forceinline__ void chain_wait(uint64_t* bar, uint32_t parity, bool& ok) {
  if (ok && !__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity))) ok = warp_wait(bar, parity);
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

// Two FP32 values as BF16 hi and lo halves.
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
  hi = *reinterpret_cast<const uint32_t*>(&b);
  const float2 d = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), make_float2(-1.f, -1.f), x);
  const __nv_bfloat162 c = __floats2bfloat162_rn(d.x, d.y);
  lo = *reinterpret_cast<const uint32_t*>(&c);
}

// Eight of them.
__device__ __forceinline__ void split8(const float* x, uint4& hi, uint4& lo) {
  split2(make_float2(x[0], x[1]), hi.x, lo.x);
  split2(make_float2(x[2], x[3]), hi.y, lo.y);
  split2(make_float2(x[4], x[5]), hi.z, lo.z);
  split2(make_float2(x[6], x[7]), hi.w, lo.w);
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
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld8_async(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 16 values of a lane as 8 + 8 columns of the operands hi and lo.
__device__ __forceinline__ void put_split16(uint32_t hi_addr, uint32_t lo_addr, const float* x) {
  uint32_t hi[8], lo[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) split2(make_float2(x[2 * j], x[2 * j + 1]), hi[j], lo[j]);
  tmem_st8(hi_addr, hi);
  tmem_st8(lo_addr, lo);
}

// D[tmem] (+)= A[tmem] * B[smem]^T, issued by one thread; 16 k are 8 columns of A.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

constexpr int kDv = 32;  // value columns of a narrow CTA
constexpr int kThinDv = 16, kThinnestDv = 8;  // and of the thin ones

// Operand tiles [hi | lo] of DV + DV value columns: piece `piece` of line `row`.
template <int DV>
__device__ __forceinline__ uint8_t* tile16(uint8_t* tile, int row, int piece) {
  const int turn = DV == 32 ? row & 7 : DV == 16 ? (row >> 1) & 3 : (row >> 2) & 1;
  return tile + row * 4 * DV + ((piece ^ turn) << 4);
}
template <int DV>
__device__ __forceinline__ uint64_t tile_desc(uint8_t* tile) {
  if constexpr (DV == 32)
    return tc::sw128_desc_mn(tc::smem_u32(tile), 0);
  else
    return tc::sw_desc_mn<2 * DV>(tc::smem_u32(tile));
}

// A row's values as operand halves: columns [8 part, 8 part + 8) of the CTA's.
template <int DV>
__device__ __forceinline__ void put_split(uint8_t* tile, int row, int part, const float (&x)[8]) {
  uint4 hi, lo;
  split8(x, hi, lo);
  *reinterpret_cast<uint4*>(tile16<DV>(tile, row, part)) = hi;
  *reinterpret_cast<uint4*>(tile16<DV>(tile, row, DV / 8 + part)) = lo;
}

// A warp's 8 accumulator columns: the hi product's plus the lo product's.
template <int DV>
__device__ __forceinline__ void get_acc(uint32_t taddr, int part, float (&x)[8]) {
  uint32_t a[8], b[8];
  tmem_ld8_async(taddr + part * 8, a);
  tmem_ld8_async(taddr + DV + part * 8, b);
  wait_ld(a);
  wait_ld(b);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 s = add2(make_float2(__uint_as_float(a[j]), __uint_as_float(a[j + 1])),
                          make_float2(__uint_as_float(b[j]), __uint_as_float(b[j + 1])));
    x[j] = s.x;
    x[j + 1] = s.y;
  }
}

// The same for a token-row accumulator, 16 rows in the fragment layout: rows
// lane / 4 and + 8, columns 2 (lane % 4) and + 1.
__device__ __forceinline__ void ld_frag8(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
template <int DV>
__device__ __forceinline__ void get_rows(uint32_t taddr, int part, float2 (&x)[2]) {
  uint32_t a[4], b[4];
  ld_frag8(taddr + part * 8, a);
  ld_frag8(taddr + DV + part * 8, b);
  wait_ld(a);
  wait_ld(b);
#pragma unroll
  for (int e = 0; e < 2; ++e)
    x[e] = add2(make_float2(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1])),
                make_float2(__uint_as_float(b[2 * e]), __uint_as_float(b[2 * e + 1])));
}
template <int DV>
__device__ __forceinline__ void put_rows(uint8_t* tile, int row, int part, int lane, const float2 (&x)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint32_t hi, lo;
    split2(x[e], hi, lo);
    const int at = 4 * (lane & 3);
    *reinterpret_cast<uint32_t*>(tile16<DV>(tile, row + 8 * e, part) + at) = hi;
    *reinterpret_cast<uint32_t*>(tile16<DV>(tile, row + 8 * e, DV / 8 + part) + at) = lo;
  }
}

// The chain warps have written an operand: the warps that issue its products
// wait for them at a hardware barrier, which wakes them sooner than an mbarrier
// would and costs the chain one instruction.  kBarSq: S, for Q S.
// A barrier counts arrivals, whoever they come from: one ahead of its phase would
// count for another warp, and the issuing warp would be left at a later phase for
// good.  What keeps a chain warp from that is its waits for products; one that has
// run out of time skips those, and waits at the barriers instead.  kBarPast keeps
// the two issuing warps within a chunk of each other, so that who has met one at
// S knows the other to be past D of the chunk before.  By then it is, long since,
// unless a wait has run out.
enum { kBarS = 2, kBarY = 3, kBarDs = 4, kBarD = 5, kBarSq = 6, kBarPast = 7 };
template <int WARPS>
__device__ __forceinline__ void barrier_arrive(int id, bool ok) {
  if (ok)
    asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "n"(32 * (WARPS + 1)) : "memory");
  else
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(32 * (WARPS + 1)) : "memory");
}
template <bool TMEM, int WARPS>
__device__ __forceinline__ void chain_arrive(int id, bool ok) {
  if (TMEM) wait_st();
  tc::tc_fence_before();
  barrier_arrive<WARPS>(id, ok);
}
// For operands in shared memory the fence between the chain's writes and the
// tensor core's reads stands here, behind the barrier, in the issuing warp alone:
// in front of it, in every chain warp, it took about 280 cycles of each stage.
template <bool TMEM, int WARPS>
__device__ __forceinline__ void chain_await(int id) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(32 * (WARPS + 1)) : "memory");
  if (!TMEM) tc::fence_async_smem();
  tc::tc_fence_after();
}

__device__ __forceinline__ void past_arrive() { asm volatile("barrier.cta.arrive %0, 64;" ::"r"(static_cast<int>(kBarPast)) : "memory"); }
__device__ __forceinline__ void past_await() { asm volatile("barrier.cta.sync %0, 64;" ::"r"(static_cast<int>(kBarPast)) : "memory"); }

__device__ __forceinline__ int64_t seq_start(const GdnPrefillArgs& a, int n) {
  return a.cu_seqlens ? (int64_t)a.cu_seqlens[n] : a.total_tokens / a.num_seqs * n;
}
// Tokens of sequence n, -1 where its bounds are not those of a sequence.
__device__ __forceinline__ int seq_len(const GdnPrefillArgs& a, int n) {
  const int64_t t0 = seq_start(a, n), t1 = seq_start(a, n + 1);
  const bool bad = t0 < 0 || t1 < t0 || t1 > a.total_tokens || (n == 0 && t0 != 0) ||
                   (n == a.num_seqs - 1 && t1 != a.total_tokens);
  return bad ? -1 : (int)(t1 - t0);
}
__device__ __forceinline__ int seq_chunks(const GdnPrefillArgs& a, int n) {
  const int len = seq_len(a, n);
  return len > 0 ? (len + kC - 1) / kC : 0;
}

// Fragments of 16 x 16 (or 8 x 16) pieces of 128-byte-swizzled BF16 tiles for
// the register-to-register products of the inversion, which are too small and
// too close together for a trip through TMEM.
__device__ __forceinline__ uint32_t elem_addr(const uint8_t* tile, int row, int col) {
  return tc::smem_u32(tile) + row * 128 + (((col >> 3) ^ (row & 7)) << 4) + (col & 7) * 2;
}
__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Left operand: rows [r0, r0 + 16), columns [k0, k0 + 16) of the tile.
__device__ __forceinline__ void frag_left(const uint8_t* tile, int r0, int k0, int lane, uint32_t (&f)[4]) {
  ldm4(elem_addr(tile, r0 + (lane & 15), k0 + 8 * (lane >> 4)), f);
}
// Left operand, the transpose of rows [k0, k0 + 16), columns [m0, m0 + 16).
__device__ __forceinline__ void frag_left_t(const uint8_t* tile, int k0, int m0, int lane, uint32_t (&f)[4]) {
  ldm4t(elem_addr(tile, k0 + (lane & 7) + 8 * (lane >> 4), m0 + (lane & 8)), f);
}
// Right operand, the transpose of rows [n0, n0 + 16), columns [k0, k0 + 16):
// {f0, f1} for n0.., {f2, f3} for n0 + 8...
__device__ __forceinline__ void frag_right_t(const uint8_t* tile, int n0, int k0, int lane, uint32_t (&f)[4]) {
  ldm4(elem_addr(tile, n0 + (lane & 7) + 8 * (lane >> 4), k0 + (lane & 8)), f);
}
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One warp: 16 rows [r0, ..) and 16 columns [c0, ..) of -T22 (A21 T11), KB blocks
// of 16 in the middle (rows and columns of T11 from k0, rows of A21 and of T22
// from l0).  T11 is lower triangular, so the blocks above column block c0 are
// skipped, and those of T22 right of row block r0.  (A21 T11)^T comes out of the
// first products in the layout in which the second ones take it.  Every factor
// is a BF16 pair; lo lo is left out (2^-18).
template <int KB>
__device__ __forceinline__ void inverse_block(uint8_t* t_hi, uint8_t* t_lo, const uint8_t* a_hi, const uint8_t* a_lo,
                                              int k0, int l0, int r0, int c0, int lane) {
  float z[2 * KB][4];
#pragma unroll
  for (int i = 0; i < 2 * KB; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) z[i][e] = 0.f;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int k = k0 + 16 * kb;
    if (k < c0) continue;
    uint32_t th[4], tl[4];
    frag_left_t(t_hi, k, c0, lane, th);
    frag_left_t(t_lo, k, c0, lane, tl);
#pragma unroll
    for (int ib = 0; ib < KB; ++ib) {
      if (l0 + 16 * ib > r0) continue;  // rows that T22's row block does not use
      uint32_t ah[4], al[4];
      frag_right_t(a_hi, l0 + 16 * ib, k, lane, ah);
      frag_right_t(a_lo, l0 + 16 * ib, k, lane, al);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        mma16(z[2 * ib + p], th, al[2 * p], al[2 * p + 1]);
        mma16(z[2 * ib + p], tl, ah[2 * p], ah[2 * p + 1]);
        mma16(z[2 * ib + p], th, ah[2 * p], ah[2 * p + 1]);
      }
    }
  }
  float w[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) w[i][e] = 0.f;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int k = l0 + 16 * kb;
    if (k > r0) continue;
    uint32_t th[4], tl[4];
    frag_left(t_hi, r0, k, lane, th);
    frag_left(t_lo, r0, k, lane, tl);
#pragma unroll
    for (int p = 0; p < 2; ++p) {  // columns c0 + 8 p ..
      uint32_t h0, l0_, h1, l1;
      split2(make_float2(z[2 * kb][2 * p], z[2 * kb][2 * p + 1]), h0, l0_);
      split2(make_float2(z[2 * kb + 1][2 * p], z[2 * kb + 1][2 * p + 1]), h1, l1);
      mma16(w[p], th, l0_, l1);
      mma16(w[p], tl, h0, h1);
      mma16(w[p], th, h0, h1);
    }
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t hi, lo;
      split2(make_float2(-w[p][2 * e], -w[p][2 * e + 1]), hi, lo);
      const int row = r0 + (lane >> 2) + 8 * e, col = c0 + 8 * p + 2 * (lane & 3);
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(elem_addr(t_hi, row, col)), "r"(hi) : "memory");
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(elem_addr(t_lo, row, col)), "r"(lo) : "memory");
    }
}

// T = (Diag(1 / beta) + A)^-1 by blocks, 128 threads, into the tiles t_hi, t_lo
// (whose blocks above the diagonal are zero already): diagonal blocks of 16 by
// forward substitution in FP32, x_i = beta_i (e_i - sum_(j < i) A_ij x_j), one
// warp each and a column per lane; then T21 = -T22 A21 T11 for blocks of 16 and
// of 32.  diag: FP32 diagonal blocks of A.
__device__ __forceinline__ void invert64(uint8_t* t_hi, uint8_t* t_lo, const uint8_t* a_hi, const uint8_t* a_lo,
                                         const float* diag, const float* beta, int warp, int lane) {
  {
    const float* d = diag + warp * 16 * kLdG;
    const int col = lane & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float4 row[4];
#pragma unroll
      for (int j = 0; j < (i + 3) / 4; ++j) row[j] = *reinterpret_cast<const float4*>(d + i * kLdG + 4 * j);
      const float* r = reinterpret_cast<const float*>(row);
      float s0 = col == i ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) {
        if (j & 1) s1 = fmaf(-r[j], x[j], s1); else s0 = fmaf(-r[j], x[j], s0);
      }
      x[i] = beta[16 * warp + i] * (s0 + s1);
    }
    uint8_t* tile = lane < 16 ? t_hi : t_lo;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint16_t hi, lo;
      tc::split_bf16(x[i], hi, lo);
      asm volatile("st.shared.b16 [%0], %1;" ::"r"(elem_addr(tile, 16 * warp + i, 16 * warp + col)),
                   "h"(lane < 16 ? hi : lo)
                   : "memory");
    }
  }
  __syncthreads();
  if (warp < 2)
    inverse_block<1>(t_hi, t_lo, a_hi, a_lo, 32 * warp, 32 * warp + 16, 32 * warp + 16, 32 * warp, lane);
  __syncthreads();
  inverse_block<2>(t_hi, t_lo, a_hi, a_lo, 0, 32, 32 + 16 * (warp >> 1), 16 * (warp & 1), lane);
}

// K rows [len, 64) zeroed by `threads` threads: they belong to the next sequence
// or lie past the last token, and NaN times a zero factor is NaN.  The two halves
// of 64 channels are `half` bytes apart.
__device__ __forceinline__ void zero_rows(uint8_t* k, int half, int len, int t, int threads) {
  for (int x = t; x < (kC - len) * 16; x += threads)
    *line16(k + (x & 1) * half, len + x / 16, (x >> 1) & 7) = make_uint4(0, 0, 0, 0);
}

template <bool F16>
__global__ void __launch_bounds__(128, ChunkCfg::kCtas)
    gdn_chunk_kernel(const GdnPrefillArgs args, const __grid_constant__ GdnMaps maps) {
  using C = ChunkCfg;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBar);  // rows landed, [K; Q] K^T done, TMEM address
  const int t = threadIdx.x, quad = t >> 5, lane = t & 31;
  grid_dependency_launch();
  if (tc::smem_u32(smem) & 1023u) {  // swizzled tiles start on 1024 bytes
    if (t == 0) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
    return;
  }
  // what needs nothing of the chunk comes before the walk that finds it
  const int h = blockIdx.x % args.HV, id = blockIdx.x / args.HV;
  const ScalarGateArgs& ga = args.gate;
  const float a_log = ga.A_log ? ga.A_log[h] : 0.f;
  const float bias = ga.dt_bias ? ga.dt_bias[h] : 0.f;
  uint8_t* kq = smem;
  if (quad == 0) tc::tmem_alloc(reinterpret_cast<uint32_t*>(&bars[2]), C::kTmCols);
  if (t == 0) {
    tc::mbar_init(&bars[0], 1);
    tc::mbar_init(&bars[1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // whoever waits for this kernel waits for the one that splits FP16 rows too
  auto after_split = [] {
    if constexpr (F16) grid_dependency_wait();
  };
  auto leave = [&] {  // no chunk here: the grid is an upper bound
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (quad == 0) tc::tmem_dealloc(*reinterpret_cast<const uint32_t*>(&bars[2]), C::kTmCols);
    after_split();
  };
  // the chunk's sequence: every warp walks over the sequences, 128 at a time
  int n = -1, c = 0;
  for (int n0 = 0, base = 0; n0 < args.num_seqs && n < 0; n0 += 128) {
    int cnt[4], sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = n0 + 4 * lane + e;
      cnt[e] = m < args.num_seqs ? seq_chunks(args, m) : 0;
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
      n = n0 + 4 * src + __shfl_sync(0xffffffffu, mine, src);
      c = id - __shfl_sync(0xffffffffu, at, src);
    }
    base += __shfl_sync(0xffffffffu, run, 31);
  }
  if (n < 0) {
    leave();
    return;
  }
  // (a sequence without a state slot gets records too, which none reads: to ask would cost each CTA a load's wait)
  const int64_t t0 = seq_start(args, n) + (int64_t)c * kC;
  const int left = seq_len(args, n) - c * kC, len = left < kC ? left : kC;
  if (t == 0) {
    tc::mbar_expect_tx(&bars[0], C::kRowBytes);
    const int tok = (int)t0, hk = h / args.G;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      tma_box(kq + a * 16384, &maps.k, a * 64, hk, tok, &bars[0]);
      tma_box(kq + a * 16384 + 8192, &maps.q, a * 64, hk, tok, &bars[0]);
    }
  }

  uint8_t* rec = args.records + ((int64_t)id * args.HV + h) * kRecBytes;
  uint8_t* a_hi = smem;  // over the two halves of K
  uint8_t* a_lo = smem + 16384;
  uint8_t* t_hi = smem + 8192;  // over the two halves of Q
  uint8_t* t_lo = smem + 24576;
  float* diag = reinterpret_cast<float*>(smem + C::kDiag);
  float* c_hi = reinterpret_cast<float*>(smem + C::kGate);  // c_i = c_hi + c_lo (first the log-decays)
  float* c_lo = c_hi + kC;
  float* beta_s = c_lo + kC;
  float* rks = beta_s + kC;
  ChunkScalars& sc = *reinterpret_cast<ChunkScalars*>(smem + C::kScalars);
  if (t < kC) {  // log-decay and beta of a token; past the end nothing decays and nothing is written
    float g = 0.f, b = 0.f;
    if (t < len) {
      const int64_t at = (t0 + t) * args.HV + h;
      b = in16_to_float<F16>(args.beta[at]);
      g = scalar_log_decay<F16>(ga, scalar_gate_load(ga, args.a, at), -expf(a_log), bias);
      b = ga.beta_is_raw ? sigmoidf_(b) : b;
    }
    c_hi[t] = g;
    beta_s[t] = b;
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(&bars[2]);
  const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16);
  // c_i, the running sums of the log-decays, as pairs hi + lo (two-sum): their
  // differences count.  Every warp scans all 64, two a lane.
  float2 c_i, c_mid, c_last;
  {
    auto plus = [](float2 a, float2 b) {
      const float s = a.x + b.x, z = s - a.x;
      return make_float2(s, a.y + (((a.x - (s - z)) + (b.x - z)) + b.y));
    };
    const float2 g = *reinterpret_cast<const float2*>(c_hi + 2 * lane);
    float2 run = plus(make_float2(g.x, 0.f), make_float2(g.y, 0.f));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float2 up = make_float2(__shfl_up_sync(0xffffffffu, run.x, d), __shfl_up_sync(0xffffffffu, run.y, d));
      if (lane >= d) run = plus(up, run);
    }
    const float2 even = plus(run, make_float2(-g.y, 0.f));  // token 2 lane; run: token 2 lane + 1
    auto from = [](float2 x, int l) {
      return make_float2(__shfl_sync(0xffffffffu, x.x, l), __shfl_sync(0xffffffffu, x.y, l));
    };
    const int i = 32 * (quad & 1) + lane;
    const float2 a = from(even, i >> 1), b = from(run, i >> 1);
    c_i = i & 1 ? b : a;
    c_mid = from(even, kC / 4);
    c_last = from(run, 31);
    __syncthreads();  // every warp has read the log-decays
    if (quad == 0) {
      *reinterpret_cast<float2*>(c_hi + 2 * lane) = make_float2(even.x, run.x);
      *reinterpret_cast<float2*>(c_lo + 2 * lane) = make_float2(even.y, run.y);
    }
  }
  bool bad = !warp_wait(&bars[0], 0);
  if (len < kC) {
    zero_rows(kq, 16384, len, t, 128);
    tc::fence_async_smem();
    __syncthreads();
  }
  if (quad == 0 && !bad && elect_one()) {  // [K; Q] K^T
    constexpr uint32_t kIdA = F16 ? tc::idesc_f16_f32(128, 64) : tc::idesc_bf16_f32(128, 64);
    const uint64_t op = tc::sw128_desc(tc::smem_u32(kq));
    tc::tc_fence_after();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t off = ((j >> 2) * 16384 + (j & 3) * 32) >> 4;
      tc::mma_bf16(tmem, op + off, op + off, kIdA, j > 0);
    }
    tc::mma_commit(&bars[1]);
  }
  __syncwarp();
  const bool krow = quad < 2;
  const int i = 32 * (quad & 1) + lane;  // token of the chunk
  const int row = krow ? i : 64 + i;  // row of [K; Q]
  float2 ss[4];  // four running sums, for latency
#pragma unroll
  for (int e = 0; e < 4; ++e) ss[e] = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int a = 0; a < 2; ++a)
#pragma unroll 4
    for (int p = 0; p < 8; ++p) {
      const uint4 w = *line16(kq + a * 16384, row, p);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float f0 = __uint_as_float(ww[e] << 16), f1 = __uint_as_float(ww[e] & 0xffff0000u);
        if (F16) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[e]));
          f0 = f.x;
          f1 = f.y;
        }
        ss[e] = fma2(make_float2(f0, f1), make_float2(f0, f1), ss[e]);
      }
    }
  const float sq = ((ss[0].x + ss[0].y) + (ss[1].x + ss[1].y)) + ((ss[2].x + ss[2].y) + (ss[3].x + ss[3].y));
  const float r = (krow ? 1.f : ga.scale) * (ga.use_qk_l2norm ? rsqrtf(sq + kNormEps) : 1.f);
  // r_i r_j e^(c_i - c_j) as a product of row and column factors about the
  // middle of the chunk, where those stay in FP32's range; term by term otherwise
  const float ci_hi = c_i.x, ci_lo = c_i.y;
  const float mid = (ci_hi - c_mid.x) + (ci_lo - c_mid.y);
  const bool far = !(fabsf(mid) <= 60.f);
  if (krow) rks[i] = r * expf(-mid);
  bad |= !warp_wait(&bars[1], 0);
  const bool wide = __syncthreads_or(far);
  if (wide) {
    if (krow) rks[i] = r;
    __syncthreads();
  }
  for (int x = t; x < 1024; x += 128)  // blocks of T above the diagonal are not written below
    reinterpret_cast<uint4*>(x < 512 ? t_hi : t_lo)[x & 511] = make_uint4(0, 0, 0, 0);
  tc::tc_fence_after();
  const float ei = expf(ci_hi + ci_lo);
  const float ui = wide ? r : r * expf(mid);
  const float si = krow && i < len ? r * expf((c_last.x - ci_hi) + (c_last.y - ci_lo)) : 0.f;
  const int top = 32 * (quad & 1) + 31;  // last row of this warp
#pragma unroll 1
  for (int jb = 0; jb < 4; ++jb) {
    float d[16];
    if (16 * jb <= top) {
      tc::tmem_ld16(acc + 16 * jb, d);
      float f[16];
#pragma unroll
      for (int e = 0; e < 4; ++e) *reinterpret_cast<float4*>(f + 4 * e) = *reinterpret_cast<const float4*>(rks + 16 * jb + 4 * e);
      if (wide) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          f[e] *= expf((ci_hi - c_hi[16 * jb + e]) + (ci_lo - c_lo[16 * jb + e]));
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int j = 16 * jb + e;
        d[e] = (krow ? j < i : j <= i) ? (ui * f[e]) * d[e] : 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) d[e] = 0.f;
    }
    if (krow) {
      if (jb < (i >> 4)) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint4 hi, lo;
          split8(d + 8 * p, hi, lo);
          *line16(a_hi, i, 2 * jb + p) = hi;
          *line16(a_lo, i, 2 * jb + p) = lo;
        }
      } else if (jb == (i >> 4)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<float4*>(diag + i * kLdG + 4 * e) =
              make_float4(d[4 * e], d[4 * e + 1], d[4 * e + 2], d[4 * e + 3]);
      }
    } else {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint4 hi, lo;
        split8(d + 8 * p, hi, lo);
        *line16(rec + kRecP, i, 2 * jb + p) = hi;  // global memory
        *line16(rec + kRecPlo, i, 2 * jb + p) = lo;
      }
    }
  }
  tc::tc_fence_before();
  bad = __syncthreads_or(bad);
  if (quad == 0 && !bad) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, C::kTmCols);
  }
  invert64(t_hi, t_lo, a_hi, a_lo, diag, beta_s, quad, lane);
  if (krow) {
    sc.a[i] = -r * ei;
    sc.s[i] = si;
    if (i == 63) {
      sc.last = ei;
      sc.done = bad ? 0.f : 1.f;
    }
  } else {
    sc.o[i] = r * ei;
  }
  tc::fence_async_smem();
  __syncthreads();
  if (t == 0) {
    if (bad) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
    tc::bulk_s2g(rec + kRecT, t_hi, 8192);
    tc::bulk_s2g(rec + kRecTlo, t_lo, 8192);
    tc::bulk_s2g(rec + kRecScalars, &sc, 1024);
    tc::bulk_commit();
    tc::bulk_wait_read();
  }
  if (bad && quad == 0) {  // a wait ran out: once more, with its limit, for rows and products under way
    warp_wait(&bars[0], 0);
    warp_wait(&bars[1], 0);
    tc::tc_fence_after();
    tc::tmem_dealloc(*reinterpret_cast<const uint32_t*>(&bars[2]), C::kTmCols);
  }
  after_split();
}

// What a state CTA works on.
struct Unit {
  int h, slice, n;
  int columns;  // value columns: kThinnestDv, kThinDv, kDv, or kHeadDim in the wide form
  int L, nch, slot;
  int64_t t0;
};

// Microseconds / 20 of a state CTA: measured, 16 heads, BF16.
__device__ __forceinline__ int64_t narrow_time(int64_t chunks) { return 29 * chunks + 120; }
__device__ __forceinline__ int64_t wide_time(int64_t chunks) { return 62 * chunks + 200; }

// Which unit a state CTA takes; false: none is left.  CTAs start in order, so
// the longest sequences come first.  In the mixed kernel the k longest ones take
// the narrow form; every CTA finds the k of the least estimate of the whole: the
// longest CTA, and, where not all start at once, all CTAs' time over the SMs and
// the last one behind it.  Wide CTAs beside narrow ones slow these down, by a
// twelfth in the estimate.  All narrow, all wide (both in kernels of their own)
// and the choice, whole call, 16 heads (us): 8087 and seven shorter of 16980 tokens
// 256, 407, 260; 8 x 4096 506, 308, 314; 8000 and 20 x 200 239, 389, 249; 64 x 512
// 569, 354, 367; 8000 and 20 x 1000, L2 cold, 459, 484, 351.
template <int kForm>
__device__ __forceinline__ bool pick_unit(const GdnPrefillArgs& args, uint8_t* smem, Unit& s) {
  constexpr int kCols = kForm == kThinnest ? kThinnestDv : kForm == kThin ? kThinDv : kDv, kSlices = kHeadDim / kCols;
  const int tid = threadIdx.x, seqs = args.num_seqs;
  int narrow = kForm == kWide || kForm == kMixed ? 0 : seqs;
  int* order = reinterpret_cast<int*>(smem);
  if (kForm == kMixed || args.longest_first) {
    int* len_s = order + kMaxSorted;
    int* chunks = len_s + kMaxSorted;
    unsigned long long* best = reinterpret_cast<unsigned long long*>(chunks + kMaxSorted);
    if (tid < seqs) len_s[tid] = seq_len(args, tid);
    if (tid == 0) *best = ~0ull;
    __syncthreads();
    if (tid < seqs) {
      const int mine = len_s[tid];
      int before = 0;
      for (int m = 0; m < seqs; ++m) before += len_s[m] > mine || (len_s[m] == mine && m < tid);
      order[before] = tid;
      chunks[before] = mine > 0 ? (mine + kC - 1) / kC : 0;
    }
    __syncthreads();
    if (kForm == kMixed) {
      if (tid <= seqs && (tid <= args.most_narrow || (tid == seqs && args.all_narrow))) {
        const int64_t k = tid;
        int64_t in_narrow = 0, all = 0;
        for (int m = 0; m < seqs; ++m) {
          in_narrow += m < tid ? chunks[m] : 0;
          all += chunks[m];
        }
        int64_t cost = 0;
        if (args.HV * (kSlices * k + seqs - k) > args.sms) {
          const int64_t sum = kSlices * (narrow_time(in_narrow) + narrow_time(0) * (k - 1)) +
                              wide_time(all - in_narrow) + wide_time(0) * (seqs - k - 1);
          cost = args.HV * sum / args.sms + (k < seqs ? wide_time(chunks[seqs - 1]) : narrow_time(chunks[seqs - 1]));
        }
        if (k > 0) cost = max(cost, narrow_time(chunks[0]));
        if (k < seqs) cost = max(cost, wide_time(chunks[k]));
        if (k > 0 && k < seqs) cost += cost / 12;
        atomicMin(best, (unsigned long long)cost << 8 | (unsigned)tid);
      }
      __syncthreads();
      narrow = (int)(*best & 255);
    }
  }
  int b = blockIdx.x;
  if (b < narrow * kSlices * args.HV) {
    s.columns = kCols;
    s.slice = b % kSlices;
    s.h = b / kSlices % args.HV;
    s.n = b / kSlices / args.HV;
  } else {
    b -= narrow * kSlices * args.HV;
    s.columns = kHeadDim;
    s.slice = 0;
    s.h = b % args.HV;
    s.n = narrow + b / args.HV;
  }
  const bool some = s.n < seqs;
  if (kForm == kMixed || args.longest_first) {
    if (some) s.n = order[s.n];
    __syncthreads();  // the lists lie where rows land
  }
  if (!some) grid_dependency_wait();  // as in begin_unit
  return some;
}

// The first steps of a state CTA: refusals (false: the whole CTA leaves),
// barriers and TMEM.
__device__ __forceinline__ bool begin_unit(const GdnPrefillArgs& args, uint8_t* smem, Bars& bars, Unit& s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool reporter = tid == 0 && s.h == 0 && s.slice == 0;
  const int n = s.n;
  const int L = seq_len(args, n);
  const int slot = args.state_idx[n];
  bool stop = L <= 0;
  if (L < 0 && reporter) set_error(args.err_flag, KDA_DEVERR_SEQLENS);
  if (L > 0 && (slot < 0 || slot >= args.pool_slots)) {  // padding or out of range: zero outputs, no state touched
    stop = true;
    if (slot != -1 && reporter) set_error(args.err_flag, KDA_DEVERR_SLOT);
    const int64_t t0 = seq_start(args, n);
    const int pieces = s.columns / 8;
    for (int64_t i = tid; i < (int64_t)L * pieces; i += kStateThreads)
      *reinterpret_cast<uint4*>(args.o + ((t0 + i / pieces) * args.HV + s.h) * kHeadDim + s.slice * s.columns +
                                (i % pieces) * 8) = make_uint4(0, 0, 0, 0);
  }
  if (tc::smem_u32(smem) & 1023u) {  // swizzled tiles start on 1024 bytes
    stop = true;
    if (tid == 0) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
  }
  if (warp == 1) {  // record of this sequence's first chunk
    int64_t id = 0;
    for (int m = lane; m < n; m += 32) id += seq_chunks(args, m);
#pragma unroll
    for (int m = 16; m; m >>= 1) id += __shfl_xor_sync(0xffffffffu, id, m);
    if (lane == 0) bars.chunk0 = id;
  }
  __syncthreads();
  s.t0 = seq_start(args, n);
  s.L = L;
  s.slot = slot;
  s.nch = (L + kC - 1) / kC;
  if (!stop && bars.chunk0 + s.nch > args.max_chunks) {  // overlapping sequences have more chunks than tokens allow
    stop = true;
    if (reporter) set_error(args.err_flag, KDA_DEVERR_SEQLENS);
  }
  if (stop) {
    grid_dependency_wait();  // whoever waits for this kernel waits for the one before too
    return false;
  }

  tc::fence_async_smem();  // lists lay where rows land
  if (warp == kMmaWarp) tc::tmem_alloc(&bars.tmem, kTmCols);
  if (tid == 0) {
    bars.timed_out = 0;
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(&bars.key[i], 1);
      tc::mbar_init(&bars.key_free[i], 2);
      tc::mbar_init(&bars.rec[i], 1);
      tc::mbar_init(&bars.rec_free[i], 1 + kOutWarps);
    }
    tc::mbar_init(&bars.tail, 1);
    tc::mbar_init(&bars.x_full, 1);
    tc::mbar_init(&bars.xq_full, 1);
    tc::mbar_init(&bars.d_full, 1);
    tc::mbar_init(&bars.u_full, 1);
    tc::mbar_init(&bars.o_full, 1);
    tc::mbar_init(&bars.o_read, kOutWarps);
    tc::mbar_init(&bars.drained[0], 1);
    tc::mbar_init(&bars.drained[1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  return true;
}

// And its last ones.  Where a wait has run out, products may still be under way:
// their issuing warps wait for them, with a limit, before TMEM and shared memory go.
__device__ __forceinline__ void end_unit(const GdnPrefillArgs& args, Bars& bars, uint32_t tmem, bool ok) {
  if (!ok) bars.timed_out = 1;
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const int warp = threadIdx.x >> 5;
  if (bars.timed_out) {
    if (threadIdx.x == 0) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
    if (warp == kMmaWarp || warp == kSideWarp) {
      uint64_t* bar = &bars.drained[warp == kSideWarp];
      if (elect_one()) tc::mma_commit(bar);  // the same lane as issued them
      __syncwarp();
      warp_wait(bar, 0);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmCols);
}

// The row warp: every chunk's keys and queries, as two halves of 64 channels each.
template <bool F16>
__device__ __forceinline__ bool load_keys(const GdnPrefillArgs& args, const GdnMaps& maps, uint8_t* smem, Bars& bars,
                                          const Unit& s, int lane) {
  using C = Cfg<F16>;
  bool ok = true;
  const bool leader = elect_one();
  if constexpr (F16) grid_dependency_wait();
  int issued = 0;
  for (int c = 0; c < s.nch; ++c) {
    const int sl = c % C::kKeys;
    if (c >= C::kKeys && !(ok = warp_wait(&bars.key_free[sl], (uint32_t)(c / C::kKeys - 1) & 1u))) break;
    uint8_t* key = smem + sl * C::kKeyBytes;
    if (leader) {
      tc::mbar_expect_tx(&bars.key[sl], C::kKeyBytes);
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        tma_box(key + a * 8192, &maps.k, a * 64, s.h / args.G, (int)s.t0 + c * kC, &bars.key[sl]);
        tma_box(key + C::kQ + a * 8192, &maps.q, a * 64, s.h / args.G, (int)s.t0 + c * kC, &bars.key[sl]);
        if (F16) {
          tma_box(key + 16384 + a * 8192, &maps.k_lo, a * 64, s.h / args.G, (int)s.t0 + c * kC, &bars.key[sl]);
          tma_box(key + C::kQ + 16384 + a * 8192, &maps.q_lo, a * 64, s.h / args.G, (int)s.t0 + c * kC, &bars.key[sl]);
        }
      }
    }
    __syncwarp();
    issued = c + 1;
    if (c == s.nch - 1 && s.L % kC != 0) {
      if (!(ok = warp_wait(&bars.key[sl], (uint32_t)(c / C::kKeys) & 1u))) break;
      zero_rows(key, 8192, s.L % kC, lane, 32);
      if (F16) zero_rows(key + 16384, 8192, s.L % kC, lane, 32);
      tc::fence_async_smem();
      __syncwarp();
      if (leader) arrive(&bars.tail);
    }
  }
  // nothing may land after the CTA is gone
  for (int c = issued > C::kKeys ? issued - C::kKeys : 0; c < issued; ++c)
    warp_wait(&bars.key[c % C::kKeys], (uint32_t)(c / C::kKeys) & 1u);
  return ok;
}

// The record warp.
template <bool F16>
__device__ __forceinline__ bool load_records(const GdnPrefillArgs& args, uint8_t* smem, Bars& bars, const Unit& s) {
  using C = Cfg<F16>;
  bool ok = true;
  const bool leader = elect_one();
  grid_dependency_wait();
  const uint8_t* src = args.records + (bars.chunk0 * args.HV + s.h) * kRecBytes;
  int issued = 0;
  for (int c = 0; c < s.nch; ++c) {
    const int sl = c % C::kRecs;
    if (c >= C::kRecs && !(ok = warp_wait(&bars.rec_free[sl], (uint32_t)(c / C::kRecs - 1) & 1u))) break;
    if (leader) {
      tc::mbar_expect_tx(&bars.rec[sl], kRecBytes);
      tc::bulk_g2s(smem + C::kRec + sl * kRecBytes, src + (int64_t)c * args.HV * kRecBytes, kRecBytes, &bars.rec[sl]);
    }
    __syncwarp();
    issued = c + 1;
  }
  for (int c = issued > C::kRecs ? issued - C::kRecs : 0; c < issued; ++c)
    warp_wait(&bars.rec[c % C::kRecs], (uint32_t)(c / C::kRecs) & 1u);
  return ok;
}

// The narrow and the thin form: DV value columns.
template <bool F16, int DV>
__device__ __forceinline__ void narrow_unit(const GdnPrefillArgs& args, const GdnMaps& maps, uint8_t* smem, Bars& bars,
                                            const Unit& s) {
  using C = Cfg<F16>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = s.h, L = s.L, nch = s.nch;
  const int64_t t0 = s.t0;
  const uint32_t tmem = bars.tmem;
  bool ok = true;
  constexpr int kParts = DV / 8, kWarps = 4 * kParts;  // chain warps
  if (warp < kWarps) {
    // ---------------------------------------------------------------- chain
    // A warp that runs out of time goes on without waiting, so that the others
    // still meet it.
    const int quad = warp & 3, part = warp >> 2;
    const int row = 16 * quad + (lane >> 2);  // token rows row and row + 8 of the chunk, columns
    const int colx = s.slice * DV + part * 8 + 2 * (lane & 3);  // colx and colx + 1 of those
    const int dk = 32 * quad + lane;          // key channel of the state,
    const int col0 = s.slice * DV + part * 8;  // its columns col0 ..
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    float* root = args.pool + (((size_t)s.slot * args.HV + h) * kHeadDim + col0) * kHeadDim + dk;
    float S[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) S[j] = root[j * kHeadDim];
    const int64_t cid = bars.chunk0;
    uint32_t vraw[2];
    const int64_t vstep = (int64_t)args.HV * kHeadDim;
    const kda_bf16* vsrc = args.v + ((t0 + row) * args.HV + h) * kHeadDim + colx;
    auto load_v = [&](int c) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        vraw[e] = c * kC + row + 8 * e < L ? __ldg(reinterpret_cast<const uint32_t*>(vsrc + 8 * e * vstep)) : 0u;
      vsrc += kC * vstep;
    };
    load_v(0);
    for (int c = 0; c < nch; ++c) {
      const int sl = c % C::kRecs;
      const uint32_t cp = (uint32_t)c & 1u;
      put_split<DV>(smem + C::kS, dk, part, S);
      chain_arrive<false, kWarps>(kBarS, ok);
      barrier_arrive<kWarps>(kBarSq, ok);
      if (args.intermediate) {
        if (cid + c < args.inter_chunks) {
          float* dst = args.intermediate + (((size_t)(cid + c) * args.HV + h) * kHeadDim + col0) * kHeadDim + dk;
#pragma unroll
          for (int j = 0; j < 8; ++j) dst[j * kHeadDim] = S[j];
        } else if (threadIdx.x == 0 && h == 0 && s.slice == 0) {
          set_error(args.err_flag, KDA_DEVERR_INTERMEDIATE);
        }
      }
      const ChunkScalars& sc = *reinterpret_cast<const ChunkScalars*>(smem + C::kRec + sl * kRecBytes + kRecScalars);
      chain_wait(&bars.rec[sl], (uint32_t)(c / C::kRecs) & 1u, ok);
      const float last = sc.last;
      const float fa[2] = {sc.a[row], sc.a[row + 8]}, fs[2] = {sc.s[row], sc.s[row + 8]};
      ok = ok && sc.done == 1.f;
      chain_wait(&bars.x_full, cp, ok);
      tc::tc_fence_after();
      float2 x[2], y[2];
      get_rows<DV>(lanes + kTmX, part, x);
      // Y = v - r e^c (K S)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float2 v;
        if constexpr (F16)
          v = __half22float2(*reinterpret_cast<const __half2*>(&vraw[e]));
        else
          v = make_float2(__uint_as_float(vraw[e] << 16), __uint_as_float(vraw[e] & 0xffff0000u));
        x[e] = fma2(make_float2(fa[e], fa[e]), x[e], v);
      }
      put_rows<DV>(smem + C::kY, row, part, lane, x);
      chain_arrive<false, kWarps>(kBarY, ok);
      if (c + 1 < nch) load_v(c + 1);
      chain_wait(&bars.d_full, cp, ok);
      tc::tc_fence_after();
      get_rows<DV>(lanes + kTmX, part, x);
#pragma unroll
      for (int e = 0; e < 2; ++e) y[e] = mul2(make_float2(fs[e], fs[e]), x[e]);
      put_rows<DV>(smem + C::kY, row, part, lane, y);
      chain_arrive<false, kWarps>(kBarDs, ok);
      put_rows<DV>(smem + C::kD, row, part, lane, x);
      chain_arrive<false, kWarps>(kBarD, ok);
      chain_wait(&bars.u_full, cp, ok);
      tc::tc_fence_after();
      float u[8];
      get_acc<DV>(lanes + kTmU, part, u);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 n2 = fma2(make_float2(last, last), make_float2(S[j], S[j + 1]), make_float2(u[j], u[j + 1]));
        S[j] = n2.x;
        S[j + 1] = n2.y;
      }
    }
    if (ok)
#pragma unroll
      for (int j = 0; j < 8; ++j) root[j * kHeadDim] = S[j];
  } else if (warp >= kChainWarps && warp < kMmaWarp) {
    // --------------------------------------------------------------- outputs
    // O = scale rq e^c Q S + P D, 16 token rows a warp.
    const int quad = warp & 3;
    const int row = 16 * quad + (lane >> 2);
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    kda_bf16* dst = args.o + ((t0 + row) * args.HV + h) * kHeadDim + s.slice * DV + 2 * (lane & 3);
    const int64_t step = (int64_t)args.HV * kHeadDim;
    for (int c = 0; c < nch; ++c, dst += kC * step) {
      const int sl = c % C::kRecs;
      const ChunkScalars& sc = *reinterpret_cast<const ChunkScalars*>(smem + C::kRec + sl * kRecBytes + kRecScalars);
      if (!(ok = warp_wait(&bars.rec[sl], (uint32_t)(c / C::kRecs) & 1u))) break;
      const float fo[2] = {sc.o[row], sc.o[row + 8]};
      __syncwarp();
      if (lane == 0) arrive(&bars.rec_free[sl]);
      if (!(ok = warp_wait(&bars.o_full, (uint32_t)c & 1u))) break;
      tc::tc_fence_after();
      uint32_t w[kParts][2];
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        float2 x[2], u[2];
        get_rows<DV>(lanes + kTmQ, part, x);
        get_rows<DV>(lanes + kTmO, part, u);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 y = fma2(make_float2(fo[e], fo[e]), x[e], u[e]);
          w[part][e] = pack_out16x2<F16>(y.x, y.y);
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(&bars.o_read);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (c * kC + row + 8 * e < L) {
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            *reinterpret_cast<uint32_t*>(dst + 8 * e * step + 8 * part) = w[part][e];
        }
    }
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------- the chain's products
    // As the chain warps, it goes on without waiting once out of time.
    constexpr uint32_t kId64 = tc::idesc_bf16_f32(64, 2 * DV) | tc::kIdescMnB;
    constexpr uint32_t kIdU = tc::idesc_bf16_f32(128, 2 * DV) | tc::kIdescMnA | tc::kIdescMnB;
    const uint64_t s_op = tile_desc<DV>(smem + C::kS);
    const uint64_t y_op = tile_desc<DV>(smem + C::kY);
    const bool leader = elect_one();
    for (int c = 0; c < nch; ++c) {
      const int ks = c % C::kKeys, sl = c % C::kRecs;
      const uint32_t key = tc::smem_u32(smem + ks * C::kKeyBytes);
      const uint64_t k_op = tc::sw128_desc(key), kl_op = tc::sw128_desc(key + 16384);
      const uint64_t kt_op = tc::sw128_desc_mn(key, 8192), klt_op = tc::sw128_desc_mn(key + 16384, 8192);
      const uint64_t t_op = tc::sw128_desc(tc::smem_u32(smem + C::kRec + sl * kRecBytes));
      ok = ok && warp_wait(&bars.key[ks], (uint32_t)(c / C::kKeys) & 1u);
      if (c == nch - 1 && L % kC != 0) ok = ok && warp_wait(&bars.tail, 0);
      if (c > 0) past_await();
      chain_await<false, kWarps>(kBarS);
      if (leader && ok) {  // X = K S
#pragma unroll
        for (int b = 0; b < (F16 ? 2 : 1); ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc::mma_bf16(tmem + kTmX, (b ? kl_op : k_op) + (((j >> 2) * 8192 + (j & 3) * 32) >> 4), s_op + ((j * 64 * DV) >> 4),
                         kId64, b + j > 0);
        tc::mma_commit(&bars.x_full);
      }
      __syncwarp();
      ok = ok && warp_wait(&bars.rec[sl], (uint32_t)(c / C::kRecs) & 1u);
      // behind D, the chain overwrites what P D of the last chunk reads
      if (c > 0) ok = ok && warp_wait(&bars.o_full, (uint32_t)(c - 1) & 1u);
      chain_await<false, kWarps>(kBarY);
      if (leader && ok) {  // D = T Y
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmX, t_op + (((b ? kRecTlo : 0) + j * 32) >> 4), y_op + ((j * 64 * DV) >> 4), kId64, b + j > 0);
        tc::mma_commit(&bars.d_full);
      }
      __syncwarp();
      chain_await<false, kWarps>(kBarDs);
      if (leader && ok) {  // dS = K^T D'
#pragma unroll
        for (int b = 0; b < (F16 ? 2 : 1); ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmU, (b ? klt_op : kt_op) + ((j * 2048) >> 4), y_op + ((j * 64 * DV) >> 4), kIdU, b + j > 0);
        tc::mma_commit(&bars.key_free[ks]);
      }
      __syncwarp();
      // behind dS, the chain overwrites what Q S reads
      ok = ok && warp_wait(&bars.xq_full, (uint32_t)c & 1u);
      if (leader && ok) tc::mma_commit(&bars.u_full);
      __syncwarp();
    }
    past_await();
  } else if (warp == kSideWarp) {
    // ----------------------------------------- products for the output alone
    // As the chain warps, it goes on without waiting once out of time.
    constexpr uint32_t kId64 = tc::idesc_bf16_f32(64, 2 * DV) | tc::kIdescMnB;
    const uint64_t s_op = tile_desc<DV>(smem + C::kS);
    const uint64_t d_op = tile_desc<DV>(smem + C::kD);
    const bool leader = elect_one();
    for (int c = 0; c < nch; ++c) {
      const int ks = c % C::kKeys, sl = c % C::kRecs;
      const uint32_t rec = tc::smem_u32(smem + C::kRec + sl * kRecBytes);
      const uint64_t q_op = tc::sw128_desc(tc::smem_u32(smem + ks * C::kKeyBytes + C::kQ)), p_op = tc::sw128_desc(rec + kRecP);
      ok = ok && warp_wait(&bars.key[ks], (uint32_t)(c / C::kKeys) & 1u);
      ok = ok && warp_wait(&bars.rec[sl], (uint32_t)(c / C::kRecs) & 1u);
      if (c > 0) ok = ok && warp_wait(&bars.o_read, (uint32_t)(c - 1) & 1u);
      chain_await<false, kWarps>(kBarSq);
      if (leader && ok) {  // Q S
#pragma unroll
        for (int b = 0; b < (F16 ? 2 : 1); ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc::mma_bf16(tmem + kTmQ, q_op + ((b * 16384 + (j >> 2) * 8192 + (j & 3) * 32) >> 4), s_op + ((j * 64 * DV) >> 4),
                         kId64, b + j > 0);
        tc::mma_commit(&bars.xq_full);
        tc::mma_commit(&bars.key_free[ks]);
      }
      __syncwarp();
      chain_await<false, kWarps>(kBarD);  // the chain is also past T and this chunk's scalars
      past_arrive();
      if (leader && ok) {  // P D
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmO, p_op + (((b ? kRecPlo - kRecP : 0) + j * 32) >> 4), d_op + ((j * 64 * DV) >> 4), kId64,
                         b + j > 0);
        tc::mma_commit(&bars.o_full);
        tc::mma_commit(&bars.rec_free[sl]);
      }
      __syncwarp();
    }
  } else if (warp == kKeyWarp) {
    ok = load_keys<F16>(args, maps, smem, bars, s, lane);
  } else if (warp == kRecWarp) {
    ok = load_records<F16>(args, smem, bars, s);
  }
  end_unit(args, bars, tmem, ok);
}

// The wide form: all value columns, transposed.
template <bool F16>
__device__ __forceinline__ void wide_unit(const GdnPrefillArgs& args, const GdnMaps& maps, uint8_t* smem, Bars& bars,
                                          const Unit& s) {
  using C = Cfg<F16>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = s.h, L = s.L, nch = s.nch;
  const int64_t t0 = s.t0;
  const uint32_t tmem = bars.tmem;
  bool ok = true;
  if (warp < kChainWarps) {
    // 768 threads start with 80 registers each; 512 at 96, 128 at 56 and 128 at 40 are those 61440
    asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    // ---------------------------------------------------------------- chain
    // A warp that runs out of time goes on without waiting, so that the others
    // still meet it.
    const int quad = warp & 3, part = warp >> 2;
    const int dv = 32 * quad + lane;  // this thread's value column
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    const int tok0 = 16 * part;       // its tokens of a chunk; its key channels of the state: 32 part ..
    float* root = args.pool + (((size_t)s.slot * args.HV + h) * kHeadDim + dv) * kHeadDim + 32 * part;
    float S[32];
#pragma unroll
    for (int j = 0; j < 8; ++j) *reinterpret_cast<float4*>(S + 4 * j) = *reinterpret_cast<const float4*>(root + 4 * j);
    const int64_t cid = bars.chunk0;
    // v of the 16 tokens.  A lane loads two neighbouring columns of every other
    // token and trades with its neighbour: 32-bit loads, two tokens a register.
    const int64_t vstep = (int64_t)args.HV * kHeadDim;
    const int odd = lane & 1;
    const uint32_t pick = odd ? 0x3276u : 0x5410u;
    const kda_bf16* vsrc = args.v + ((t0 + tok0 + odd) * args.HV + h) * kHeadDim + (dv & ~1);
    uint32_t vraw[8];
    auto load_v = [&](int c) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        vraw[j] = c * kC + tok0 + odd + 2 * j < L ? __ldg(reinterpret_cast<const uint32_t*>(vsrc + 2 * j * vstep)) : 0u;
      vsrc += kC * vstep;
    };
    load_v(0);
    for (int c = 0; c < nch; ++c) {
      const int sl = c % C::kRecs;
      const uint32_t cp = (uint32_t)c & 1u;
      put_split16(lanes + kTmS + 16 * part, lanes + kTmSlo + 16 * part, S);
      put_split16(lanes + kTmS + 16 * part + 8, lanes + kTmSlo + 16 * part + 8, S + 16);
      chain_arrive<true, kChainWarps>(kBarS, ok);
      barrier_arrive<kChainWarps>(kBarSq, ok);
      if (args.intermediate) {
        if (cid + c < args.inter_chunks) {
          float* dst = args.intermediate + (((size_t)(cid + c) * args.HV + h) * kHeadDim + dv) * kHeadDim + 32 * part;
#pragma unroll
          for (int j = 0; j < 8; ++j) *reinterpret_cast<float4*>(dst + 4 * j) = *reinterpret_cast<const float4*>(S + 4 * j);
        } else if (threadIdx.x == 0 && h == 0) {
          set_error(args.err_flag, KDA_DEVERR_INTERMEDIATE);
        }
      }
      uint32_t v2[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v2[j] = __byte_perm(vraw[j], __shfl_xor_sync(0xffffffffu, vraw[j], 1), pick);
      const ChunkScalars& sc = *reinterpret_cast<const ChunkScalars*>(smem + C::kRec + sl * kRecBytes + kRecScalars);
      chain_wait(&bars.rec[sl], (uint32_t)(c / C::kRecs) & 1u, ok);
      const float last = sc.last;
      ok = ok && sc.done == 1.f;
      chain_wait(&bars.x_full, cp, ok);
      tc::tc_fence_after();
      float x[16];
      {
        uint32_t r[16];
        tc::tmem_ld16_async(lanes + kTmX + tok0, r);
        wait_ld(r);
        // Y = v - r e^c (K S)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 a = *reinterpret_cast<const float2*>(sc.a + tok0 + 2 * j);
          float2 v;
          if constexpr (F16)
            v = __half22float2(*reinterpret_cast<const __half2*>(&v2[j]));
          else
            v = make_float2(__uint_as_float(v2[j] << 16), __uint_as_float(v2[j] & 0xffff0000u));
          const float2 y = fma2(a, make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), v);
          x[2 * j] = y.x;
          x[2 * j + 1] = y.y;
        }
      }
      put_split16(lanes + kTmY + 8 * part, lanes + kTmYlo + 8 * part, x);
      chain_arrive<true, kChainWarps>(kBarY, ok);
      if (c + 1 < nch) load_v(c + 1);
      chain_wait(&bars.d_full, cp, ok);
      tc::tc_fence_after();
      {
        uint32_t r[16];
        tc::tmem_ld16_async(lanes + kTmX + tok0, r);
        wait_ld(r);
        float y[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[2 * j] = __uint_as_float(r[2 * j]);
          x[2 * j + 1] = __uint_as_float(r[2 * j + 1]);
          const float2 s = mul2(*reinterpret_cast<const float2*>(sc.s + tok0 + 2 * j), make_float2(x[2 * j], x[2 * j + 1]));
          y[2 * j] = s.x;
          y[2 * j + 1] = s.y;
        }
        put_split16(lanes + kTmY + 8 * part, lanes + kTmYlo + 8 * part, y);
      }
      chain_arrive<true, kChainWarps>(kBarDs, ok);
      put_split16(lanes + kTmX + tok0, lanes + kTmX + tok0 + 8, x);  // over this warp's quarter of D
      chain_arrive<true, kChainWarps>(kBarD, ok);
      chain_wait(&bars.u_full, cp, ok);
      tc::tc_fence_after();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t r[16];
        tc::tmem_ld16_async(lanes + kTmU + 32 * part + 16 * g, r);
        wait_ld(r);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 s = fma2(make_float2(last, last), make_float2(S[16 * g + j], S[16 * g + j + 1]),
                                make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])));
          S[16 * g + j] = s.x;
          S[16 * g + j + 1] = s.y;
        }
      }
    }
    if (ok)
#pragma unroll
      for (int j = 0; j < 8; ++j) *reinterpret_cast<float4*>(root + 4 * j) = *reinterpret_cast<const float4*>(S + 4 * j);
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // --------------------------------------------------------------- outputs
    // O = scale rq e^c Q S + P D, 32 value columns a warp, 64 tokens a thread.
    const int quad = warp & 3, odd = lane & 1;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t pick = odd ? 0x3276u : 0x5410u;
    const int64_t step = (int64_t)args.HV * kHeadDim;
    kda_bf16* dst = args.o + ((t0 + odd) * args.HV + h) * kHeadDim + ((32 * quad + lane) & ~1);
    for (int c = 0; c < nch; ++c, dst += kC * step) {
      const int sl = c % C::kRecs;
      const ChunkScalars& sc = *reinterpret_cast<const ChunkScalars*>(smem + C::kRec + sl * kRecBytes + kRecScalars);
      if (!(ok = warp_wait(&bars.rec[sl], (uint32_t)(c / C::kRecs) & 1u))) break;
      if (!(ok = warp_wait(&bars.o_full, (uint32_t)c & 1u))) break;
      tc::tc_fence_after();
      const int left = L - c * kC - odd;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t w[16];  // two tokens of one column each
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int tok = 32 * half + 8 * g;
          uint32_t q[8], r[8];
          tmem_ld8_async(lanes + kTmQ + tok, q);
          tmem_ld8_async(lanes + kTmO + tok, r);
          wait_ld(q);
          wait_ld(r);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = fma2(*reinterpret_cast<const float2*>(sc.o + tok + 2 * j),
                                  make_float2(__uint_as_float(q[2 * j]), __uint_as_float(q[2 * j + 1])),
                                  make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])));
            w[4 * g + j] = pack_out16x2<F16>(y.x, y.y);
          }
        }
        if (half) {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            arrive(&bars.rec_free[sl]);
            arrive(&bars.o_read);
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {  // traded for two columns of one token each
          const int tok = 32 * half + 2 * j;
          const uint32_t x = __byte_perm(w[j], __shfl_xor_sync(0xffffffffu, w[j], 1), pick);
          if (tok < left) *reinterpret_cast<uint32_t*>(dst + tok * step) = x;
        }
      }
    }
  } else if (warp == kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    // ----------------------------------------------------- the chain's products
    // As the chain warps, it goes on without waiting once out of time.
    constexpr uint32_t kId64 = tc::idesc_bf16_f32(128, 64);
    constexpr uint32_t kIdU = tc::idesc_bf16_f32(128, 128) | tc::kIdescMnB;
    const bool leader = elect_one();
    for (int c = 0; c < nch; ++c) {
      const int ks = c % C::kKeys, sl = c % C::kRecs;
      const uint32_t key = tc::smem_u32(smem + ks * C::kKeyBytes);
      const uint64_t k_op = tc::sw128_desc(key), kl_op = tc::sw128_desc(key + 16384);
      const uint64_t kt_op = tc::sw128_desc_mn(key, 8192), klt_op = tc::sw128_desc_mn(key + 16384, 8192);
      const uint64_t t_op = tc::sw128_desc(tc::smem_u32(smem + C::kRec + sl * kRecBytes));
      ok = ok && warp_wait(&bars.key[ks], (uint32_t)(c / C::kKeys) & 1u);
      if (c == nch - 1 && L % kC != 0) ok = ok && warp_wait(&bars.tail, 0);
      if (c > 0) ok = ok && warp_wait(&bars.o_full, (uint32_t)(c - 1) & 1u);  // X takes the place of the last D
      if (c > 0) past_await();
      chain_await<true, kChainWarps>(kBarS);
      if (leader && ok) {  // X^T = S^T K^T
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_ts(tmem + kTmX, tmem + (b ? kTmSlo : kTmS) + 8 * j, k_op + (((j >> 2) * 8192 + (j & 3) * 32) >> 4), kId64,
                   b + j > 0);
        if constexpr (F16) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_ts(tmem + kTmX, tmem + kTmS + 8 * j, kl_op + (((j >> 2) * 8192 + (j & 3) * 32) >> 4), kId64, true);
        }
        tc::mma_commit(&bars.x_full);
      }
      __syncwarp();
      ok = ok && warp_wait(&bars.rec[sl], (uint32_t)(c / C::kRecs) & 1u);
      chain_await<true, kChainWarps>(kBarY);
      if (leader && ok) {  // D^T = Y^T T^T: hi hi, lo hi, hi lo
#pragma unroll
        for (int b = 0; b < 3; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_ts(tmem + kTmX, tmem + (b == 1 ? kTmYlo : kTmY) + 8 * j, t_op + (((b == 2 ? kRecTlo : 0) + j * 32) >> 4),
                   kId64, b + j > 0);
        tc::mma_commit(&bars.d_full);
      }
      __syncwarp();
      chain_await<true, kChainWarps>(kBarDs);
      if (leader && ok) {  // dS^T = D'^T K
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_ts(tmem + kTmU, tmem + (b ? kTmYlo : kTmY) + 8 * j, kt_op + ((j * 2048) >> 4), kIdU, b + j > 0);
        if constexpr (F16) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_ts(tmem + kTmU, tmem + kTmY + 8 * j, klt_op + ((j * 2048) >> 4), kIdU, true);
        }
        tc::mma_commit(&bars.key_free[ks]);
      }
      __syncwarp();
      // behind dS, the chain overwrites what Q S reads
      ok = ok && warp_wait(&bars.xq_full, (uint32_t)c & 1u);
      if (leader && ok) tc::mma_commit(&bars.u_full);
      __syncwarp();
    }
    past_await();
  } else if (warp == kSideWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    // ----------------------------------------- products for the output alone
    // As the chain warps, it goes on without waiting once out of time.
    constexpr uint32_t kId64 = tc::idesc_bf16_f32(128, 64);
    const bool leader = elect_one();
    for (int c = 0; c < nch; ++c) {
      const int ks = c % C::kKeys, sl = c % C::kRecs;
      const uint32_t rec = tc::smem_u32(smem + C::kRec + sl * kRecBytes);
      const uint64_t q_op = tc::sw128_desc(tc::smem_u32(smem + ks * C::kKeyBytes + C::kQ)), p_op = tc::sw128_desc(rec + kRecP);
      ok = ok && warp_wait(&bars.key[ks], (uint32_t)(c / C::kKeys) & 1u);
      ok = ok && warp_wait(&bars.rec[sl], (uint32_t)(c / C::kRecs) & 1u);
      if (c > 0) ok = ok && warp_wait(&bars.o_read, (uint32_t)(c - 1) & 1u);
      chain_await<true, kChainWarps>(kBarSq);
      if (leader && ok) {  // S^T Q^T
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_ts(tmem + kTmQ, tmem + (b ? kTmSlo : kTmS) + 8 * j, q_op + (((j >> 2) * 8192 + (j & 3) * 32) >> 4), kId64,
                   b + j > 0);
        if constexpr (F16) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_ts(tmem + kTmQ, tmem + kTmS + 8 * j, q_op + ((16384 + (j >> 2) * 8192 + (j & 3) * 32) >> 4), kId64, true);
        }
        tc::mma_commit(&bars.xq_full);
        tc::mma_commit(&bars.key_free[ks]);
      }
      __syncwarp();
      chain_await<true, kChainWarps>(kBarD);  // the chain is also past T and this chunk's scalars
      past_arrive();
      if (leader && ok) {  // D^T P^T
#pragma unroll
        for (int b = 0; b < 3; ++b)  // hi hi, lo hi, hi lo
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_ts(tmem + kTmO, tmem + kTmX + 16 * j + (b == 1 ? 8 : 0), p_op + (((b == 2 ? kRecPlo - kRecP : 0) + j * 32) >> 4),
                   kId64, b + j > 0);
        tc::mma_commit(&bars.o_full);
        tc::mma_commit(&bars.rec_free[sl]);
      }
      __syncwarp();
    }
  } else if (warp == kKeyWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    ok = load_keys<F16>(args, maps, smem, bars, s, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    ok = load_records<F16>(args, smem, bars, s);
  }
  end_unit(args, bars, tmem, ok);
}

template <bool F16, int kForm>
__global__ void __launch_bounds__(kStateThreads, 1)
    gdn_state_kernel(const GdnPrefillArgs args, const __grid_constant__ GdnMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + Cfg<F16>::kBars);
  Unit s;
  if (!pick_unit<kForm>(args, smem, s) || !begin_unit(args, smem, bars, s)) return;
  if (kForm == kThinnest)
    narrow_unit<F16, kThinnestDv>(args, maps, smem, bars, s);
  else if (kForm == kThin)
    narrow_unit<F16, kThinDv>(args, maps, smem, bars, s);
  else if (kForm == kNarrow || (kForm == kMixed && s.columns == kDv))
    narrow_unit<F16, kDv>(args, maps, smem, bars, s);
  else
    wide_unit<F16>(args, maps, smem, bars, s);
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

// FP16 q and k as operands of the state kernel: two BF16 halves whose sum they
// are.  One 16-byte piece of each a thread.
__global__ void __launch_bounds__(256) split_rows_kernel(const uint4* __restrict__ q, const uint4* __restrict__ k,
                                                         int64_t n, uint4* q_hi, uint4* q_lo, uint4* k_hi, uint4* k_lo) {
  grid_dependency_launch();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  auto split = [i](const uint4& w, uint4* hi, uint4* lo) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = in16_to_float<true>((uint16_t)(e & 1 ? a[e / 2] >> 16 : a[e / 2] & 0xffffu));
    split8(f, hi[i], lo[i]);
  };
  const uint4 wq = __ldg(q + i), wk = __ldg(k + i);
  split(wq, q_hi, q_lo);
  split(wk, k_hi, k_lo);
}

template <bool F16, int kForm>
constexpr int kStateSmem = kForm == kWide ? Cfg<F16>::kWideSmem : Cfg<F16>::kSmem;

template <typename Kernel>
bool allow_smem(Kernel kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}
template <bool F16, int... kForms>
bool allow_forms() {
  return allow_smem(gdn_chunk_kernel<F16>, ChunkCfg::kSmem) &&
         (allow_smem(gdn_state_kernel<F16, kForms>, kStateSmem<F16, kForms>) && ...);
}
// The kernels' shared-memory limits, all of them in the first call on a device:
// a later one may be under capture.
kda_status allow_all() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_CUDA;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
    if (!allow_forms<false, kThinnest, kThin, kNarrow, kWide, kMixed>() ||
        !allow_forms<true, kThinnest, kThin, kNarrow, kWide, kMixed>())
      return KDA_ERR_CUDA;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  return KDA_OK;
}

template <bool F16>
kda_status launch_chunks(const GdnPrefillArgs& a, const GdnMaps& m, cudaStream_t st) {
  static_assert(ChunkCfg::kCtas * (ChunkCfg::kSmem + 1024) <= 233472, "CTAs per SM");
  const int64_t grid = a.max_chunks * a.HV;
  if (grid > INT32_MAX) return KDA_ERR_SHAPE;
  return launch_dependent(gdn_chunk_kernel<F16>, (unsigned)grid, 128, ChunkCfg::kSmem, F16, st, a, m);
}

template <bool F16, int kForm>
kda_status launch_state(const GdnPrefillArgs& a, const GdnMaps& m, int64_t grid, cudaStream_t st) {
  using C = Cfg<F16>;
  static_assert(C::kSmem <= 232448 && C::kWideSmem <= C::kSmem && kStateThreads == 768, "shared memory and registers");
  if (grid > INT32_MAX) return KDA_ERR_SHAPE;
  return launch_dependent(gdn_state_kernel<F16, kForm>, (unsigned)grid, kStateThreads, kStateSmem<F16, kForm>,
                          !stage_between(), st, a, m);
}

// As thin as lets all CTAs start at once: 1 x 4096 tokens, 16 heads, thin 95.5 us,
// narrow 115; 8 heads, thinnest 78, thin 84, narrow 104.  All narrow where that
// fills the SMs twice at most: compiled by itself it spills no register, so that
// 1000, 333, 77 and 2001 FP16 tokens, 16 heads, take 89 us, in the mixed kernel 101
// (4 x 1024, the other way: 74, 71).  Otherwise what the CTAs settle, since the
// lengths are on the device.  All wide where there are too many sequences to rank,
// or so many heads that narrow CTAs could not pay: they take 1.9 times as much of
// the SMs, and CTAs that find no unit (as many as the launch has beyond those of
// the choice) cost a microsecond each.
template <bool F16>
kda_status launch_states(GdnPrefillArgs a, const GdnMaps& m, cudaStream_t st) {
  const int64_t heads = (int64_t)a.num_seqs * a.HV, slices = kHeadDim / kDv;
  a.sms = sm_count();
  if (a.sms <= 0) return KDA_ERR_CUDA;
  if (heads * (kHeadDim / kThinnestDv) <= a.sms)
    return launch_state<F16, kThinnest>(a, m, heads * (kHeadDim / kThinnestDv), st);
  if (heads * (kHeadDim / kThinDv) <= a.sms) return launch_state<F16, kThin>(a, m, heads * (kHeadDim / kThinDv), st);
  if (heads * slices <= 2 * a.sms) {
    a.longest_first = a.num_seqs <= kMaxSorted && heads * slices > a.sms;
    return launch_state<F16, kNarrow>(a, m, heads * slices, st);
  }
  a.all_narrow = 2 * heads < 3 * a.sms;
  a.most_narrow = (int)(a.sms / (slices * a.HV));
  a.longest_first = a.num_seqs <= kMaxSorted && heads > a.sms;
  if (a.num_seqs > kMaxSorted || (!a.all_narrow && a.most_narrow == 0)) return launch_state<F16, kWide>(a, m, heads, st);
  const int64_t most = a.all_narrow ? a.num_seqs : a.most_narrow;
  return launch_state<F16, kMixed>(a, m, heads + most * (slices - 1) * a.HV, st);
}

int64_t most_chunks(int num_seqs, int64_t total_tokens) { return total_tokens / kC + num_seqs; }

size_t split_bytes(const kda_dims& d, int64_t total_tokens) {  // a half of q or k as BF16
  return d.dtype == KDA_DTYPE_F16 ? ((size_t)total_tokens * d.H * kHeadDim * 2 + 255) / 256 * 256 : 0;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_gdn_prefill_workspace_size(kda_dims dims, int num_seqs, int64_t total_tokens) {
  if (num_seqs < 0 || total_tokens < 0 || dims.H <= 0 || dims.HV <= 0) return 0;
  if (total_tokens > INT32_MAX) return SIZE_MAX;  // refused; no capacity check may pass
  return 4 * split_bytes(dims, total_tokens) + (size_t)most_chunks(num_seqs, total_tokens) * dims.HV * kRecBytes;
}

extern "C" kda_status kda_gdn_prefill(kda_dims dims, kda_scalar_gate gate, const kda_bf16* q, const kda_bf16* k,
                                      const kda_bf16* v, const void* a, const kda_bf16* beta, int64_t gb_rows,
                                      float* state_pool, int pool_slots, const int32_t* state_idx,
                                      const int32_t* cu_seqlens, int num_seqs, int64_t total_tokens, kda_bf16* o,
                                      float* intermediate, int64_t intermediate_chunks, void* workspace,
                                      size_t workspace_bytes, int32_t* err_flag, void* stream) {
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
  const size_t need = kda_gdn_prefill_workspace_size(dims, num_seqs, total_tokens);
  if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KDA_ERR_ALIGNMENT;
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f16 = dims.dtype == KDA_DTYPE_F16;
  const size_t part = split_bytes(dims, total_tokens);
  char* ws = static_cast<char*>(workspace);
  args.records = reinterpret_cast<uint8_t*>(ws + 4 * part);
  args.max_chunks = most_chunks(num_seqs, total_tokens);
  GdnMaps rows{}, m{};  // of the chunk kernel, which takes q and k as they are, and of the state kernel
  if (!encode_half_rows(&rows.q, q, dims.H, total_tokens) || !encode_half_rows(&rows.k, k, dims.H, total_tokens))
    return KDA_ERR_CUDA;
  m = rows;
  if (f16 && (!encode_half_rows(&m.q, ws, dims.H, total_tokens) || !encode_half_rows(&m.q_lo, ws + part, dims.H, total_tokens) ||
              !encode_half_rows(&m.k, ws + 2 * part, dims.H, total_tokens) ||
              !encode_half_rows(&m.k_lo, ws + 3 * part, dims.H, total_tokens)))
    return KDA_ERR_CUDA;
  s = allow_all();
  if (s != KDA_OK) return s;
  record_stage(0, st);
  if (f16) {
    const int64_t n = total_tokens * dims.H * (kHeadDim / 8);
    split_rows_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(
        reinterpret_cast<const uint4*>(q), reinterpret_cast<const uint4*>(k), n, reinterpret_cast<uint4*>(ws),
        reinterpret_cast<uint4*>(ws + part), reinterpret_cast<uint4*>(ws + 2 * part),
        reinterpret_cast<uint4*>(ws + 3 * part));
    s = launch_status();
    if (s != KDA_OK) return s;
  }
  s = f16 ? launch_chunks<true>(args, rows, st) : launch_chunks<false>(args, rows, st);
  if (s != KDA_OK) return s;
  record_stage(1, st);
  s = f16 ? launch_states<true>(args, m, st) : launch_states<false>(args, m, st);
  record_stage(2, st);
  return s;
}
