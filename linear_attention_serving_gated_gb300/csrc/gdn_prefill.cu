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
// The state stays on the SM for the whole sequence and no workspace goes
// through memory.  A CTA owns DVS value columns of one head's state; three
// dependent products a chunk are its chain, and their latency, not bytes or
// flops, bounds a long sequence, so everything else is kept off it:
//   * 16 chain warps hold S in FP32 registers and turn each product's TMEM
//     accumulator into the next one's operand; products are
//       X  = [K; Q] S     128 x DVS x 128  (Q rows ride along for O)
//       D  = T Y          rows 0..63 of [T; P] x Y
//       dS = K^T D'       128 x DVS x 64, D'_j = e^(c_last - c_j) r_j D_j
//     then P D for the output while the state is being updated, and Q S beside K S;
//   * the CTAs that own a head's columns form a cluster.  Its T and P are the
//     same for all of them, so each CTA's prep group of 4 warps builds them for
//     every (128 / DVS)-th chunk, ahead of the chain, from [K; Q] K^T (tensor
//     cores), inverts by blocks, and copies them with the chunk's row factors into
//     the other CTAs' shared memory; a warp beside it sums up the decays;
//   * 4 output warps join Q S and P D;
//   * one warp issues the chain's products, one the TMA loads, and one the
//     products that only the output needs; it also tells the CTA that fills a
//     slot next that it has been used up here.
// Y, D' and S enter as MN-major operands: a thread writes one token's (or key
// channel's) columns with 16-byte stores, never a transpose.
//
// Precision: FP32 operands are split in two BF16 halves (hi + lo, 2^-16 left)
// wherever the state depends on them: S, T, Y and D'.  K and Q are BF16 already.
// FP16 keys are split exactly (11 bits into 8 + 8) and FP16 queries rounded to
// BF16 by a pass over them before the kernel; FP16 operands would need S and D
// in FP16 halves, whose range is not the state's.  P alone is rounded to BF16 once (2^-9): it
// only enters the output, itself rounded to 16 bits.
#include <atomic>

#include "kda_host.h"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kC = 64;  // tokens per chunk
constexpr int kChainWarps = 16, kOutWarps = 4;
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
  int32_t* err_flag;
};

struct GdnMaps {
  CUtensorMap q, k, k_lo;
};

// What the chain warps read of a chunk beside T and P.
struct ChunkScalars {
  float a[kC];  // r_i e^(c_i)
  float s[kC];  // r_j e^(c_last - c_j), 0 past the sequence's end
  float o[kC];  // scale rq_i e^(c_i)
  float last;   // e^(c_last)
  float pad[3];
};
// Decays and betas of a chunk that this CTA prepares.
struct GateScalars {
  float hi[kC], lo[kC];  // c_i = hi + lo
  float beta[kC];
};

struct Bars {
  uint64_t full[2], free_[2];  // the chain's K/Q stages: landed, consumed
  uint64_t tail;               // rows past the end of the last chunk zeroed
  uint64_t p_full, a_full;     // prep: K/Q landed, [K; Q] K^T done
  uint64_t g_ready[2], g_free[2];    // its decays and betas
  uint64_t t_ready[3], p_ready[3], used[3];  // a slot's T and scalars, its P: written; all consumed by this CTA
  uint64_t slot_free;          // prep: its next slot has been consumed by every CTA
  uint64_t s_ready, x_full, xq_full, d_full, v_ready, u_full;
  uint64_t o_full, o_read;
};
struct Misc {
  uint32_t tmem;
  int timed_out;
};

template <int DVS, bool F16>
struct Cfg {
  static constexpr int kCl = kHeadDim / DVS;   // CTAs of a cluster
  // Slots of T and P.  No more than kCl: a chunk's slot is then used up before
  // the chunk that its own CTA prepares next asks for one, so that one barrier
  // counts both.
  static constexpr int kSlots = DVS == 64 || F16 ? 2 : 3;
  static constexpr int kTiles = DVS * 2 / 64;  // 64-wide operand tiles: [hi], [lo], or one [hi | lo]
  static constexpr int kStageBytes = 32768 + (F16 ? 16384 : 0);  // [K; Q], K lo
  static constexpr int kPrep = 2 * kStageBytes;                  // the prep group's K and Q
  static constexpr int kS = kPrep + kStageBytes;
  static constexpr int kSlot = kS + kTiles * 16384;
  static constexpr int kTPBytes = 16384 + 8192;  // T hi, P, T lo, then the scalars
  static constexpr int kCopyBytes = kTPBytes + (int)sizeof(ChunkScalars);
  static constexpr int kSlotBytes = 25600;
  static constexpr int kY = kSlot + kSlots * kSlotBytes;
  static constexpr int kD = kY + kTiles * 8192;
  // The prep group's A (hi, lo, diagonal blocks in FP32) lies in its K and Q,
  // which are loaded again only when T is there; T waits for its slot in memory
  // of its own, or, with FP16's larger stages, beside A.
  static constexpr int kA = kPrep;
  static constexpr int kABytes = 2 * 8192 + 4 * 16 * kLdG * 4;
  static constexpr int kT = F16 ? kPrep + 22528 : kD + kTiles * 8192;  // T hi, T lo
  static_assert(kABytes <= 22528 && (!F16 || 22528 + 16384 <= kStageBytes), "A and T beside each other");
  static constexpr int kScalars = F16 ? kD + kTiles * 8192 : kT + 16384;
  static constexpr int kBars = kSlot + kCopyBytes, kMisc = kBars + kSlotBytes;  // behind the slots' 25360 bytes
  static_assert(kCopyBytes + sizeof(Bars) <= kSlotBytes, "barriers");
  static constexpr int kGates = DVS == 64 || F16 ? 1 : 2;  // buffers of decays and betas
  static constexpr int kRk = kScalars + kGates * (int)sizeof(GateScalars);  // inverse key norms
  static constexpr int kSmem = kRk + kC * 4;
  static constexpr int kPrepWarp = kChainWarps + kOutWarps;
  static constexpr int kMmaWarp = kPrepWarp + 4, kLoadWarp = kMmaWarp + 1, kSideWarp = kMmaWarp + 2,
                       kGateWarp = kMmaWarp + 3;
  static constexpr int kThreads = (kGateWarp + 1) * 32;
  static_assert(kThreads == 896, "register split, named barriers");
};

// TMEM columns.  A2 takes the product of FP16 keys' low halves with the high
// ones, whose rows 64..127 mean nothing.
constexpr int kTmX = 0, kTmQ = 64, kTmD = 128, kTmU = 192, kTmO = 256, kTmA = 384, kTmA2 = 448, kTmCols = 512;

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

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_peer(const void* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(bar, rank)) : "memory");
}
// Shared memory of this CTA -> the same place in a peer, counted on its barrier.
__device__ __forceinline__ void copy_to_peer(const void* p, uint32_t bytes, const void* bar, uint32_t rank) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          peer_addr(p, rank)),
      "r"(tc::smem_u32(p)), "r"(bytes), "r"(peer_addr(bar, rank))
      : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// As warp_wait for a barrier that peers arrive on.
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity) {
  bool done = false;
  for (uint32_t i = 0; i < (1u << 22) && !done; ++i) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    done = r != 0;
  }
  return __all_sync(0xffffffffu, done);
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
// The chain warps have written the next product's operand: the issuing warp
// waits for them at the same hardware barrier, which wakes it sooner than an
// mbarrier would.
__device__ __forceinline__ void chain_arrive(int id) {
  tc::fence_async_smem();
  tc::tc_fence_before();
  asm volatile("barrier.cta.arrive %0, 544;" ::"r"(id) : "memory");
}
__device__ __forceinline__ void chain_await(int id) {
  asm volatile("barrier.cta.sync %0, 544;" ::"r"(id) : "memory");
  tc::tc_fence_after();
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

// A row's values as operand halves: columns [part * N, part * N + N) of the CTA's
// DVS = 4 N, in tiles [hi], [lo] 64 wide (DVS = 64) or one tile [hi | lo].
template <int DVS>
__device__ __forceinline__ void put_split(uint8_t* tiles, int tile_bytes, int row, int part, const float (&x)[DVS / 4]) {
#pragma unroll
  for (int j = 0; j < DVS / 32; ++j) {
    uint4 hi, lo;
    split8(x + 8 * j, hi, lo);
    const int piece = part * (DVS / 32) + j;
    *line16(tiles, row, piece) = hi;
    if (DVS == 64)
      *line16(tiles + tile_bytes, row, piece) = lo;
    else
      *line16(tiles, row, 4 + piece) = lo;
  }
}

__device__ __forceinline__ void tmem_ld8_async(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Waits for this thread's TMEM loads; r is not used before.
template <int M>
__device__ __forceinline__ void wait_ld(uint32_t (&r)[M]) {
  tc::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < M; ++i) asm volatile("" : "+r"(r[i]));
}

// A warp's accumulator columns of its part: 16, or 8 of the hi product plus the
// same 8 of the lo product.
template <int DVS>
__device__ __forceinline__ void get_acc(uint32_t taddr, int part, float (&x)[DVS / 4]) {
  if constexpr (DVS == 64) {
    uint32_t a[16];
    tc::tmem_ld16_async(taddr + part * 16, a);
    wait_ld(a);
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(a[j]);
  } else {
    uint32_t a[8], b[8];
    tmem_ld8_async(taddr + part * 8, a);
    tmem_ld8_async(taddr + 32 + part * 8, b);
    wait_ld(a);
    wait_ld(b);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(a[j]) + __uint_as_float(b[j]);
  }
}

__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
  hi = *reinterpret_cast<const uint32_t*>(&b);
  const __nv_bfloat162 c =
      __floats2bfloat162_rn(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
  lo = *reinterpret_cast<const uint32_t*>(&c);
}

// The same columns as operand halves (see put_split).
template <int J>
__device__ __forceinline__ void put_rows(uint8_t* tiles, int row, int part, int lane, const float (&x)[J][4]) {
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t hi, lo;
      split2(x[j][2 * e], x[j][2 * e + 1], hi, lo);
      const int rr = row + 8 * e, piece = part * J + j;
      uint8_t* line = tiles + rr * 128 + 4 * (lane & 3);
      *reinterpret_cast<uint32_t*>(line + ((piece ^ (rr & 7)) << 4)) = hi;
      if (J == 2)
        *reinterpret_cast<uint32_t*>(line + 8192 + ((piece ^ (rr & 7)) << 4)) = lo;
      else
        *reinterpret_cast<uint32_t*>(line + (((4 + piece) ^ (rr & 7)) << 4)) = lo;
    }
}

// A warp's columns of a token-row accumulator (its part of the slice), 16 rows in
// the fragment layout: rows lane / 4 and + 8, columns 8 j + 2 (lane % 4) and + 1;
// 16 columns (J = 2), or 8 of the hi product plus the same 8 of the lo product.
__device__ __forceinline__ void ld_frag8(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
template <int J>
__device__ __forceinline__ void get_rows(uint32_t taddr, int part, float (&x)[J][4]) {
  uint32_t a[4], b[4];
  ld_frag8(taddr + part * 8 * J, a);
  ld_frag8(taddr + part * 8 * J + (J == 2 ? 8 : 32), b);
  wait_ld(a);
  wait_ld(b);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[0][e] = __uint_as_float(a[e]);
    if (J == 2)
      x[J - 1][e] = __uint_as_float(b[e]);
    else
      x[0][e] += __uint_as_float(b[e]);
  }
}

__device__ __forceinline__ int64_t seq_start(const GdnPrefillArgs& a, int n) {
  return a.cu_seqlens ? (int64_t)a.cu_seqlens[n] : a.total_tokens / a.num_seqs * n;
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
// is a BF16 pair; lo lo is left out (2^-16).
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
      split2(z[2 * kb][2 * p], z[2 * kb][2 * p + 1], h0, l0_);
      split2(z[2 * kb + 1][2 * p], z[2 * kb + 1][2 * p + 1], h1, l1);
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
      split2(-w[p][2 * e], -w[p][2 * e + 1], hi, lo);
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
                                         const float* diag, const float* beta, int warp, int lane, int bar_id) {
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
  group_sync(bar_id);
  if (warp < 2)
    inverse_block<1>(t_hi, t_lo, a_hi, a_lo, 32 * warp, 32 * warp + 16, 32 * warp + 16, 32 * warp, lane);
  group_sync(bar_id);
  inverse_block<2>(t_hi, t_lo, a_hi, a_lo, 0, 32, 32 + 16 * (warp >> 1), 16 * (warp & 1), lane);
}

template <int DVS, bool F16>
__global__ void __launch_bounds__(Cfg<DVS, F16>::kThreads, 1)
    gdn_prefill_kernel(const GdnPrefillArgs args, const __grid_constant__ GdnMaps maps) {
  using C = Cfg<DVS, F16>;
  constexpr int N = DVS / 4;  // value columns per chain thread
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bars = *reinterpret_cast<Bars*>(smem + C::kBars);
  Misc& misc = *reinterpret_cast<Misc*>(smem + C::kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tc::smem_u32(smem) & 1023u) {  // swizzled tiles start on 1024 bytes
    if (tid == 0) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
    return;
  }
  const int slice = (int)cluster_rank();  // the cluster's CTAs are the slices of a head
  const int unit = blockIdx.x / C::kCl;
  const int h = unit % args.HV, n = unit / args.HV;
  const bool reporter = tid == 0 && slice == 0 && h == 0;

  const int64_t t0 = seq_start(args, n), t1 = seq_start(args, n + 1);
  if (t0 < 0 || t1 < t0 || t1 > args.total_tokens || (n == 0 && t0 != 0) ||
      (n == args.num_seqs - 1 && t1 != args.total_tokens)) {
    if (reporter) set_error(args.err_flag, KDA_DEVERR_SEQLENS);
    return;  // here and below the whole cluster returns
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

  if (warp == C::kMmaWarp) tc::tmem_alloc(&misc.tmem, kTmCols);
  if (tid == 0) {
    misc.timed_out = 0;
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.full[i], 1);
      tc::mbar_init(&bars.free_[i], 2);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      tc::mbar_init(&bars.t_ready[i], 1);
      tc::mbar_init(&bars.p_ready[i], 1);
      tc::mbar_init(&bars.used[i], 1 + kChainWarps + kOutWarps);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars.g_ready[i], 1);
      tc::mbar_init(&bars.g_free[i], 1);
    }
    tc::mbar_init(&bars.tail, 1);
    tc::mbar_init(&bars.p_full, 1);
    tc::mbar_init(&bars.a_full, 1);
    tc::mbar_init(&bars.slot_free, C::kCl);
    tc::mbar_init(&bars.s_ready, kChainWarps);
    tc::mbar_init(&bars.x_full, 1);
    tc::mbar_init(&bars.xq_full, 1);
    tc::mbar_init(&bars.o_full, 1);
    tc::mbar_init(&bars.o_read, kOutWarps);
    tc::mbar_init(&bars.d_full, 1);
    tc::mbar_init(&bars.v_ready, kChainWarps);
    tc::mbar_init(&bars.u_full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (!F16)  // blocks of T above the diagonal are never written
    for (int i = tid; i < 16384 / 16; i += C::kThreads) reinterpret_cast<uint4*>(smem + C::kT)[i] = make_uint4(0, 0, 0, 0);
  tc::fence_async_smem();
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();  // every CTA's barriers are up
  tc::tc_fence_after();
  const uint32_t tmem = misc.tmem;
  bool ok = true;
  // FP16: K and Q were split by the launch before
  if constexpr (F16) asm volatile("griddepcontrol.wait;" ::: "memory");

  auto load_rows = [&](uint8_t* kq, int c, uint64_t* bar) {
    tc::mbar_expect_tx(bar, C::kStageBytes);
    const int tok = (int)t0 + c * kC, hk = h / args.G;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      tma_box(kq + a * 16384, &maps.k, a * 64, hk, tok, bar);
      tma_box(kq + a * 16384 + 8192, &maps.q, a * 64, hk, tok, bar);
      if (F16) tma_box(kq + 32768 + a * 8192, &maps.k_lo, a * 64, hk, tok, bar);
    }
  };
  // K rows [len, 64) zeroed by `threads` threads: they belong to the next
  // sequence or lie past the last token, and NaN times a zero factor is NaN
  auto zero_tail = [&](uint8_t* kq, int len, int t, int threads) {
    for (int x = t; x < (kC - len) * 16; x += threads) {
      *line16(kq + (x & 1) * 16384, len + x / 16, (x >> 1) & 7) = make_uint4(0, 0, 0, 0);
      if (F16) *line16(kq + 32768 + (x & 1) * 8192, len + x / 16, (x >> 1) & 7) = make_uint4(0, 0, 0, 0);
    }
  };

  // 896 threads start with 72 registers each; 64, 64, 128 and 40 use 62464 of those 64512
  if (warp < kChainWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ---------------------------------------------------------------- chain
    // A warp that runs out of time goes on without waiting, so that the others
    // still meet it.
    constexpr int J = N / 8;
    const int quad = warp & 3, part = warp >> 2;
    const int row = 16 * quad + (lane >> 2);   // token rows row and row + 8 of the chunk
    const int colx = slice * DVS + part * N + 2 * (lane & 3);  // value columns colx + 8 j, + 1 of those
    const int dk = 32 * quad + lane;           // key channel of the state
    const int col0 = slice * DVS + part * N;   // value columns col0 + j of the state
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    float* root = args.pool + (((size_t)slot * args.HV + h) * kHeadDim + col0) * kHeadDim + dk;
    float S[N];
#pragma unroll
    for (int j = 0; j < N; ++j) S[j] = root[j * kHeadDim];
    int64_t cid = 0;  // record of this sequence's first chunk
    if (args.intermediate) {
      for (int m = lane; m < n; m += 32) {
        const int64_t len = seq_start(args, m + 1) - seq_start(args, m);
        cid += len > 0 ? (len + kC - 1) / kC : 0;
      }
#pragma unroll
      for (int m = 16; m; m >>= 1) cid += __shfl_xor_sync(0xffffffffu, cid, m);
    }
    uint32_t vraw[J][2];
    const int64_t vstep = (int64_t)args.HV * kHeadDim;
    const kda_bf16* vsrc = args.v + ((t0 + row) * args.HV + h) * kHeadDim + colx;
    auto load_v = [&](int c) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < J; ++j)
          vraw[j][e] = c * kC + row + 8 * e < L ? __ldg(reinterpret_cast<const uint32_t*>(vsrc + 8 * e * vstep + 8 * j)) : 0u;
      vsrc += kC * vstep;
    };
    load_v(0);
    for (int c = 0; c < nch; ++c) {
      const int sl = c % C::kSlots;
      const uint32_t cp = (uint32_t)c & 1u;
      put_split<DVS>(smem + C::kS, 16384, dk, part, S);
      chain_arrive(2);
      __syncwarp();
      if (lane == 0) arrive(&bars.s_ready);  // after chain_arrive's fences
      if (args.intermediate) {
        if (cid + c < args.inter_chunks) {
          float* dst = args.intermediate + (((size_t)(cid + c) * args.HV + h) * kHeadDim + col0) * kHeadDim + dk;
#pragma unroll
          for (int j = 0; j < N; ++j) dst[j * kHeadDim] = S[j];
        } else if (reporter) {
          set_error(args.err_flag, KDA_DEVERR_INTERMEDIATE);
        }
      }
      const ChunkScalars& sc =
          *reinterpret_cast<const ChunkScalars*>(smem + C::kSlot + sl * C::kSlotBytes + C::kTPBytes);
      ok = ok && warp_wait(&bars.t_ready[sl], (uint32_t)(c / C::kSlots) & 1u);
      const float last = sc.last;
      float fa[2] = {sc.a[row], sc.a[row + 8]}, fs[2] = {sc.s[row], sc.s[row + 8]};
      ok = ok && warp_wait(&bars.x_full, cp);
      tc::tc_fence_after();
      float x[J][4];
      get_rows<J>(lanes + kTmX, part, x);
      // Y = v - r e^c (K S)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = vraw[j][e >> 1];
          float v;
          if constexpr (F16)
            v = in16_to_float<true>((uint16_t)(e & 1 ? w >> 16 : w & 0xffffu));
          else
            v = __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
          x[j][e] = fmaf(-fa[e >> 1], x[j][e], v);
        }
      put_rows<J>(smem + C::kY, row, part, lane, x);
      chain_arrive(3);
      if (c + 1 < nch) load_v(c + 1);
      ok = ok && warp_wait(&bars.d_full, cp);
      tc::tc_fence_after();
      get_rows<J>(lanes + kTmD, part, x);
      float y[J][4];
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[j][e] = fs[e >> 1] * x[j][e];
      put_rows<J>(smem + C::kY, row, part, lane, y);
      chain_arrive(4);
      if (c > 0) ok = ok && warp_wait(&bars.o_full, cp ^ 1u);  // P D of the last chunk has read its D
      put_rows<J>(smem + C::kD, row, part, lane, x);
      warp_arrive(&bars.v_ready, lane);
      if (lane == 0) arrive(&bars.used[sl]);
      ok = ok && warp_wait(&bars.xq_full, cp);  // Q S has read S
      ok = ok && warp_wait(&bars.u_full, cp);
      tc::tc_fence_after();
      float u[N];
      get_acc<DVS>(lanes + kTmU, part, u);
#pragma unroll
      for (int j = 0; j < N; ++j) S[j] = fmaf(last, S[j], u[j]);
    }
    if (ok)
#pragma unroll
      for (int j = 0; j < N; ++j) root[j * kHeadDim] = S[j];
  } else if (warp < C::kPrepWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // --------------------------------------------------------------- outputs
    // O = scale rq e^c Q S + P D, 16 token rows a warp.
    constexpr int J = DVS / 32;
    const int quad = warp & 3;
    const int row = 16 * quad + (lane >> 2);
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    kda_bf16* dst = args.o + ((t0 + row) * args.HV + h) * kHeadDim + slice * DVS + 2 * (lane & 3);
    const int64_t step = (int64_t)args.HV * kHeadDim;
    for (int c = 0; c < nch; ++c, dst += kC * step) {
      const int sl = c % C::kSlots;
      const uint32_t cp = (uint32_t)c & 1u;
      const ChunkScalars& sc =
          *reinterpret_cast<const ChunkScalars*>(smem + C::kSlot + sl * C::kSlotBytes + C::kTPBytes);
      if (!(ok = warp_wait(&bars.t_ready[sl], (uint32_t)(c / C::kSlots) & 1u))) break;
      const float fo[2] = {sc.o[row], sc.o[row + 8]};
      __syncwarp();
      if (lane == 0) arrive(&bars.used[sl]);
      if (!(ok = warp_wait(&bars.xq_full, cp))) break;
      if (!(ok = warp_wait(&bars.o_full, cp))) break;
      tc::tc_fence_after();
      uint32_t w[4][J][2];
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        float x[J][4], u[J][4];
        get_rows<J>(lanes + kTmQ, part, x);
        get_rows<J>(lanes + kTmO, part, u);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            w[part][j][e] = pack_out16x2<F16>(fmaf(fo[e], x[j][2 * e], u[j][2 * e]),
                                              fmaf(fo[e], x[j][2 * e + 1], u[j][2 * e + 1]));
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(&bars.o_read);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (c * kC + row + 8 * e < L) {
#pragma unroll
          for (int part = 0; part < 4; ++part)
#pragma unroll
            for (int j = 0; j < J; ++j)
              *reinterpret_cast<uint32_t*>(dst + 8 * e * step + 8 * (part * J + j)) = w[part][j][e];
        }
    }
  } else if (warp < C::kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    // ----------------------------------------------------------------- prep
    const int t = tid - C::kPrepWarp * 32, quad = warp & 3;
    const int bar_id = 1;
    const bool krow = quad < 2;
    const int i = 32 * (quad & 1) + lane;  // token of the chunk
    const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16);
    uint8_t* kq = smem + C::kPrep;
    uint8_t* a_hi = smem + C::kA;
    uint8_t* a_lo = a_hi + 8192;
    uint8_t* t_hi = smem + C::kT;
    uint8_t* t_lo = t_hi + 8192;
    float* diag = reinterpret_cast<float*>(a_lo + 8192);
    float* rks = reinterpret_cast<float*>(smem + C::kRk);
    const ScalarGateArgs& ga = args.gate;
    if (t == 0 && slice < nch) load_rows(kq, slice, &bars.p_full);
    for (int c = slice, k = 0; c < nch; c += C::kCl, ++k) {
      const int sl = c % C::kSlots, gb = k % C::kGates;
      const int len = L - c * kC < kC ? L - c * kC : kC;
      const GateScalars& gs = *reinterpret_cast<const GateScalars*>(smem + C::kScalars + gb * sizeof(GateScalars));
      uint8_t* slot_s = smem + C::kSlot + sl * C::kSlotBytes;
      ChunkScalars& sc = *reinterpret_cast<ChunkScalars*>(slot_s + C::kTPBytes);
      bool bad = !warp_wait(&bars.p_full, (uint32_t)k & 1u);
      if (len < kC) {
        zero_tail(kq, len, t, 128);
        tc::fence_async_smem();
        group_sync(bar_id);
      }
      if (quad == 0 && !bad && elect_one()) {  // [K; Q] K^T
        constexpr uint32_t kIdA = tc::idesc_bf16_f32(128, 64);
        const uint64_t hi = tc::sw128_desc(tc::smem_u32(kq)), lo = tc::sw128_desc(tc::smem_u32(kq + 32768));
        tc::tc_fence_after();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t off = ((j >> 2) * 16384 + (j & 3) * 32) >> 4;
          tc::mma_bf16(tmem + kTmA, hi + off, hi + off, kIdA, j > 0);
        }
        if constexpr (F16) {  // K = hi + lo: K hi K lo^T, Q K lo^T beside, and K lo K hi^T apart
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc::mma_bf16(tmem + kTmA, hi + (((j >> 2) * 16384 + (j & 3) * 32) >> 4),
                         lo + (((j >> 2) * 8192 + (j & 3) * 32) >> 4), kIdA, true);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc::mma_bf16(tmem + kTmA2, lo + (((j >> 2) * 8192 + (j & 3) * 32) >> 4),
                         hi + (((j >> 2) * 16384 + (j & 3) * 32) >> 4), kIdA, j > 0);
        }
        tc::mma_commit(&bars.a_full);
      }
      __syncwarp();
      const int row = krow ? i : 64 + i;  // row of [K; Q]
      float2 ss[4];  // four running sums, for latency
#pragma unroll
      for (int e = 0; e < 4; ++e) ss[e] = make_float2(0.f, 0.f);
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const uint4 w = *line16(kq + a * 16384, row, p);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          uint4 w2 = make_uint4(0, 0, 0, 0);
          if (F16 && krow) w2 = *line16(kq + 32768 + a * 8192, row, p);
          const uint32_t ww2[4] = {w2.x, w2.y, w2.z, w2.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float f0 = __uint_as_float(ww[e] << 16), f1 = __uint_as_float(ww[e] & 0xffff0000u);
            if (F16) {
              f0 += __uint_as_float(ww2[e] << 16);
              f1 += __uint_as_float(ww2[e] & 0xffff0000u);
            }
            ss[e] = fma2(make_float2(f0, f1), make_float2(f0, f1), ss[e]);
          }
        }
      const float sq = ((ss[0].x + ss[0].y) + (ss[1].x + ss[1].y)) + ((ss[2].x + ss[2].y) + (ss[3].x + ss[3].y));
      const float r = (krow ? 1.f : ga.scale) * (ga.use_qk_l2norm ? rsqrtf(sq + kNormEps) : 1.f);
      bad |= !warp_wait(&bars.g_ready[gb], (uint32_t)(k / C::kGates) & 1u);
      // r_i r_j e^(c_i - c_j) as a product of row and column factors about the
      // middle of the chunk, where those stay in FP32's range; term by term otherwise
      const float ci_hi = gs.hi[i], ci_lo = gs.lo[i];
      const float mid = (ci_hi - gs.hi[kC / 2]) + (ci_lo - gs.lo[kC / 2]);
      const bool far = !(fabsf(mid) <= 60.f);
      if (krow) rks[i] = r * expf(-mid);
      bad |= !warp_wait(&bars.a_full, (uint32_t)k & 1u);
      bool wide = false;
      if (group_any(bar_id, bad || far)) {
        if (group_any(bar_id, bad)) {
          ok = false;
          break;
        }
        wide = true;
        if (krow) rks[i] = r;
        group_sync(bar_id);
      }
      if (F16) {  // T's place was under K and Q: zeros above the diagonal again
        for (int x = t; x < 16384 / 16; x += 128) reinterpret_cast<uint4*>(t_hi)[x] = make_uint4(0, 0, 0, 0);
      }
      tc::tc_fence_after();
      const float ei = __expf(ci_hi + ci_lo);
      const float ui = wide ? r : r * expf(mid);
      const float si = krow && i < len ? r * __expf((gs.hi[63] - ci_hi) + (gs.lo[63] - ci_lo)) : 0.f;
      const int top = 32 * (quad & 1) + 31;  // last row of this warp
      uint4 prow[8];  // P's row, kept until the slot is free
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        float d[16];
        if (16 * jb <= top) {
          tc::tmem_ld16(acc + kTmA + 16 * jb, d);
          if (F16 && krow) {
            float d2[16];
            tc::tmem_ld16(acc + kTmA2 + 16 * jb, d2);
#pragma unroll
            for (int e = 0; e < 16; ++e) d[e] += d2[e];
          }
          float f[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) *reinterpret_cast<float4*>(f + 4 * e) = *reinterpret_cast<const float4*>(rks + 16 * jb + 4 * e);
          if (wide) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              f[e] *= __expf((ci_hi - gs.hi[16 * jb + e]) + (ci_lo - gs.lo[16 * jb + e]));
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
          prow[2 * jb] = round8(d);
          prow[2 * jb + 1] = round8(d + 8);
        }
      }
      tc::tc_fence_before();
      group_sync(bar_id);
      invert64(t_hi, t_lo, a_hi, a_lo, diag, gs.beta, quad, lane, bar_id);
      if (!F16) {
        tc::fence_async_smem();
        group_sync(bar_id);  // A has been used: the next K and Q may land over it
        if (t == 0 && c + C::kCl < nch) load_rows(kq, c + C::kCl, &bars.p_full);
      }
      // the slot's last chunk has been used by every CTA of the cluster
      if (c >= C::kSlots)
        bad = !warp_wait_cluster(&bars.slot_free, (uint32_t)(k - (C::kSlots > slice ? 1 : 0)) & 1u);
      if (group_any(bar_id, bad)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {  // T hi and lo
        const int at = (x * 128 + t) * 16;
        *reinterpret_cast<uint4*>(slot_s + at) = *reinterpret_cast<const uint4*>(t_hi + at);
        *reinterpret_cast<uint4*>(slot_s + 16384 + at) = *reinterpret_cast<const uint4*>(t_lo + at);
      }
      if (krow) {
        sc.a[i] = r * ei;
        sc.s[i] = si;
        if (i == 63) sc.last = ei;
      } else {
        sc.o[i] = r * ei;
#pragma unroll
        for (int p = 0; p < 8; ++p) *line16(slot_s, 64 + i, p) = prow[p];
      }
      tc::fence_async_smem();
      group_sync(bar_id);  // all of the slot is written
      if (t == 0) {
        arrive(&bars.g_free[gb]);
        arrive(&bars.t_ready[sl]);
        arrive(&bars.p_ready[sl]);
        // a peer's shared memory takes about 18 bytes a clock, so what its chain
        // needs first goes first to all of them
#pragma unroll
        for (int p = 1; p < C::kCl; ++p) {
          const uint32_t to = (uint32_t)(slice + p) % C::kCl;
          copy_to_peer(slot_s, 8192, &bars.t_ready[sl], to);
          copy_to_peer(slot_s + 16384, C::kCopyBytes - 16384, &bars.t_ready[sl], to);
        }
#pragma unroll
        for (int p = 1; p < C::kCl; ++p)
          copy_to_peer(slot_s + 8192, 8192, &bars.p_ready[sl], (uint32_t)(slice + p) % C::kCl);
        if (F16 && c + C::kCl < nch) load_rows(kq, c + C::kCl, &bars.p_full);
      }
    }
  } else if (warp == C::kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    // ----------------------------------------------------- the chain's products
    // As the chain warps, it goes on without waiting once out of time.
    constexpr uint32_t kIdX = tc::idesc_bf16_f32(64, 64) | tc::kIdescMnB;
    constexpr uint32_t kIdU = tc::idesc_bf16_f32(128, 64) | tc::kIdescMnA | tc::kIdescMnB;
    const bool leader = elect_one();
    const uint64_t s_op = tc::sw128_desc_mn(tc::smem_u32(smem + C::kS), 0);
    const uint64_t y_op = tc::sw128_desc_mn(tc::smem_u32(smem + C::kY), 0);
    for (int c = 0; c < nch; ++c) {
      const int sl = c % C::kSlots, st = c & 1;
      const uint32_t kq = tc::smem_u32(smem + st * C::kStageBytes);
      const uint64_t k_op = tc::sw128_desc(kq), kl_op = tc::sw128_desc(kq + 32768);
      const uint64_t kt_op = tc::sw128_desc_mn(kq, 16384), klt_op = tc::sw128_desc_mn(kq + 32768, 8192);
      const uint64_t t_op = tc::sw128_desc(tc::smem_u32(smem + C::kSlot + sl * C::kSlotBytes));
      ok = ok && warp_wait(&bars.full[st], (uint32_t)(c >> 1) & 1u);
      if (c == nch - 1 && L % kC != 0) ok = ok && warp_wait(&bars.tail, 0);
      chain_await(2);
      if (leader && ok) {  // X = K S
#pragma unroll
        for (int b = 0; b < C::kTiles; ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc::mma_bf16(tmem + kTmX, k_op + (((j >> 2) * 16384 + (j & 3) * 32) >> 4),
                         s_op + ((b * 16384 + j * 2048) >> 4), kIdX, b + j > 0);
        if constexpr (F16) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc::mma_bf16(tmem + kTmX, kl_op + (((j >> 2) * 8192 + (j & 3) * 32) >> 4), s_op + ((j * 2048) >> 4), kIdX,
                         true);
        }
        tc::mma_commit(&bars.x_full);
      }
      __syncwarp();
      ok = ok && warp_wait(&bars.t_ready[sl], (uint32_t)(c / C::kSlots) & 1u);
      chain_await(3);
      if (leader && ok) {  // D = T Y
#pragma unroll
        for (int b = 0; b < C::kTiles; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmD, t_op + ((j * 32) >> 4), y_op + ((b * 8192 + j * 2048) >> 4), kIdX, b + j > 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tc::mma_bf16(tmem + kTmD, t_op + ((16384 + j * 32) >> 4), y_op + ((j * 2048) >> 4), kIdX, true);
        tc::mma_commit(&bars.d_full);
      }
      __syncwarp();
      chain_await(4);
      if (leader && ok) {  // dS = K^T D'
#pragma unroll
        for (int b = 0; b < C::kTiles; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmU, kt_op + ((j * 2048) >> 4), y_op + ((b * 8192 + j * 2048) >> 4), kIdU, b + j > 0);
        if constexpr (F16) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmU, klt_op + ((j * 2048) >> 4), y_op + ((j * 2048) >> 4), kIdU, true);
        }
        tc::mma_commit(&bars.u_full);
        tc::mma_commit(&bars.free_[st]);
      }
      __syncwarp();
    }
  } else if (warp == C::kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    // -------------------------------------------------------------- TMA loads
    const bool leader = elect_one();
    for (int c = 0; c < nch; ++c) {
      const int st = c & 1;
      if (c >= 2 && !(ok = warp_wait(&bars.free_[st], (uint32_t)(c / 2 - 1) & 1u))) break;
      uint8_t* kq = smem + st * C::kStageBytes;
      if (leader) load_rows(kq, c, &bars.full[st]);
      __syncwarp();
      if (c == nch - 1 && L % kC != 0) {
        if (!(ok = warp_wait(&bars.full[st], (uint32_t)(c >> 1) & 1u))) break;
        zero_tail(kq, L % kC, lane, 32);
        tc::fence_async_smem();
        __syncwarp();
        if (leader) arrive(&bars.tail);
      }
    }
  } else if (warp == C::kSideWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    // ------------------------- products for the output alone; the slots' traffic
    constexpr uint32_t kIdX = tc::idesc_bf16_f32(64, 64) | tc::kIdescMnB;
    const bool leader = elect_one();
    auto expect = [&](int c) {  // a peer's copies will land in this slot
      if (leader && c < nch && c % C::kCl != slice) {
        tc::mbar_expect_tx(&bars.t_ready[c % C::kSlots], C::kCopyBytes - 8192);
        tc::mbar_expect_tx(&bars.p_ready[c % C::kSlots], 8192);
      }
    };
    for (int c = 0; c < C::kSlots; ++c) expect(c);
    const uint64_t s_op = tc::sw128_desc_mn(tc::smem_u32(smem + C::kS), 0);
    const uint64_t d_op = tc::sw128_desc_mn(tc::smem_u32(smem + C::kD), 0);
    for (int c = 0; c < nch; ++c) {
      const int sl = c % C::kSlots, st = c & 1;
      const uint32_t cp = (uint32_t)c & 1u;
      const uint64_t q_op = tc::sw128_desc(tc::smem_u32(smem + st * C::kStageBytes + 8192));
      const uint64_t p_op = tc::sw128_desc(tc::smem_u32(smem + C::kSlot + sl * C::kSlotBytes + 8192));
      if (!(ok = warp_wait(&bars.full[st], (uint32_t)(c >> 1) & 1u))) break;
      if (!(ok = warp_wait(&bars.s_ready, cp))) break;
      if (c > 0 && !(ok = warp_wait(&bars.o_read, cp ^ 1u))) break;  // both accumulators have been read
      tc::tc_fence_after();
      if (leader) {  // Q S
#pragma unroll
        for (int b = 0; b < C::kTiles; ++b)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc::mma_bf16(tmem + kTmQ, q_op + (((j >> 2) * 16384 + (j & 3) * 32) >> 4),
                         s_op + ((b * 16384 + j * 2048) >> 4), kIdX, b + j > 0);
        tc::mma_commit(&bars.xq_full);
        tc::mma_commit(&bars.free_[st]);
      }
      __syncwarp();
      if (!(ok = warp_wait(&bars.p_ready[sl], (uint32_t)(c / C::kSlots) & 1u))) break;
      if (!(ok = warp_wait(&bars.v_ready, cp))) break;
      tc::tc_fence_after();
      if (leader) {  // P D
#pragma unroll
        for (int b = 0; b < C::kTiles; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_bf16(tmem + kTmO, p_op + ((j * 32) >> 4), d_op + ((b * 8192 + j * 2048) >> 4), kIdX,
                         b + j > 0);
        tc::mma_commit(&bars.o_full);
        tc::mma_commit(&bars.used[sl]);
      }
      __syncwarp();
      // used up here: the CTA that fills the slot next is told
      if (c + C::kSlots < nch) {
        if (!(ok = warp_wait(&bars.used[sl], (uint32_t)(c / C::kSlots) & 1u))) break;
        expect(c + C::kSlots);
        if (leader) arrive_peer(&bars.slot_free, (uint32_t)(c + C::kSlots) % C::kCl);
        __syncwarp();
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    // ------------------------------------------------------------------ gate
    const ScalarGateArgs& ga = args.gate;
    const float neg_rate = ga.A_log ? -expf(ga.A_log[h]) : 0.f;
    const float bias = ga.dt_bias ? ga.dt_bias[h] : 0.f;
    for (int c = slice, k = 0; c < nch; c += C::kCl, ++k) {
      const int gb = k % C::kGates;
      GateScalars& gs = *reinterpret_cast<GateScalars*>(smem + C::kScalars + gb * sizeof(GateScalars));
      float gl[2], be[2];  // tokens 2 lane, 2 lane + 1; past the end nothing decays and nothing is written
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = c * kC + 2 * lane + e;
        gl[e] = be[e] = 0.f;
        if (tok < L) {
          const int64_t at = (t0 + tok) * args.HV + h;
          const float b = in16_to_float<F16>(args.beta[at]);
          gl[e] = scalar_log_decay<F16>(ga, args.a, at, neg_rate, bias);
          be[e] = ga.beta_is_raw ? sigmoidf_(b) : b;
        }
      }
      // running sums in FP64, kept as two floats: differences of them count
      const double pair = (double)gl[0] + (double)gl[1];
      double run = pair;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += up;
      }
      const double c0 = run - (double)gl[1];
      if (k >= C::kGates && !(ok = warp_wait(&bars.g_free[gb], (uint32_t)(k / C::kGates - 1) & 1u))) break;
      gs.hi[2 * lane] = (float)c0;
      gs.lo[2 * lane] = (float)(c0 - (double)(float)c0);
      gs.hi[2 * lane + 1] = (float)run;
      gs.lo[2 * lane + 1] = (float)(run - (double)(float)run);
      gs.beta[2 * lane] = be[0];
      gs.beta[2 * lane + 1] = be[1];
      __syncwarp();
      if (lane == 0) arrive(&bars.g_ready[gb]);
    }
  }
  if (!ok) misc.timed_out = 1;
  tc::tc_fence_before();
  __syncthreads();
  // peers copy into this CTA's shared memory and signal its barriers
  cluster_sync();
  tc::tc_fence_after();
  if (misc.timed_out) {
    if (tid == 0) set_error(args.err_flag, KDA_DEVERR_TIMEOUT);
    // every role has stopped, but not all copies were waited for: none takes
    // this long, and none may land after the CTA is gone
    for (int i = 0; i < 4; ++i) __nanosleep(500000);
  }
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

// FP16 q and k as the BF16 operands of the kernel: keys as two halves, whose sum
// is the key, queries rounded.  One 16-byte piece of each a thread.
__global__ void __launch_bounds__(256) split_rows_kernel(const uint4* __restrict__ q, const uint4* __restrict__ k,
                                                         int64_t n, uint4* q_hi, uint4* k_hi, uint4* k_lo) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const uint4 wq = __ldg(q + i), wk = __ldg(k + i);
  const uint32_t a[4] = {wq.x, wq.y, wq.z, wq.w}, b[4] = {wk.x, wk.y, wk.z, wk.w};
  float fq[8], fk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    fq[e] = in16_to_float<true>((uint16_t)(e & 1 ? a[e / 2] >> 16 : a[e / 2] & 0xffffu));
    fk[e] = in16_to_float<true>((uint16_t)(e & 1 ? b[e / 2] >> 16 : b[e / 2] & 0xffffu));
  }
  uint4 hi, lo;
  split8(fk, hi, lo);
  q_hi[i] = round8(fq);
  k_hi[i] = hi;
  k_lo[i] = lo;
}

template <int DVS, bool F16>
kda_status launch_prefill(const GdnPrefillArgs& a, const GdnMaps& m, cudaStream_t st) {
  using C = Cfg<DVS, F16>;
  static_assert(C::kSmem <= 232448, "shared memory of one CTA");
  static_assert(C::kSlots <= C::kCl && sizeof(ChunkScalars) % 16 == 0, "slots");
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_CUDA;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
    if (cudaFuncSetAttribute(gdn_prefill_kernel<DVS, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
        cudaSuccess)
      return KDA_ERR_CUDA;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  const int64_t grid = (int64_t)a.num_seqs * a.HV * C::kCl;
  if (grid > INT32_MAX) return KDA_ERR_SHAPE;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C::kCl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // behind split_rows_kernel
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = F16 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, gdn_prefill_kernel<DVS, F16>, a, m);
  return launch_status();
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t kda_gdn_prefill_workspace_size(kda_dims dims, int64_t total_tokens) {
  if (dims.dtype != KDA_DTYPE_F16 || dims.H <= 0 || total_tokens < 0) return 0;
  if (total_tokens > INT32_MAX) return SIZE_MAX;  // refused; no capacity check may pass
  return 3 * (size_t)total_tokens * dims.H * kHeadDim * 2;
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
  const size_t need = kda_gdn_prefill_workspace_size(dims, total_tokens);
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return KDA_ERR_ALIGNMENT;
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
  const size_t part = need / 3;
  char* ws = static_cast<char*>(workspace);
  GdnMaps m{};
  if (!encode_half_rows(&m.q, f16 ? static_cast<const void*>(ws) : q, dims.H, total_tokens) ||
      !encode_half_rows(&m.k, f16 ? static_cast<const void*>(ws + part) : k, dims.H, total_tokens) ||
      (f16 && !encode_half_rows(&m.k_lo, ws + 2 * part, dims.H, total_tokens)))
    return KDA_ERR_CUDA;
  record_stage(0, st);
  if (f16) {
    const int64_t n = total_tokens * dims.H * (kHeadDim / 8);
    split_rows_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(
        reinterpret_cast<const uint4*>(q), reinterpret_cast<const uint4*>(k), n, reinterpret_cast<uint4*>(ws),
        reinterpret_cast<uint4*>(ws + part), reinterpret_cast<uint4*>(ws + 2 * part));
    s = launch_status();
    if (s != KDA_OK) return s;
  }
  record_stage(1, st);
  const int sms = sm_count();
  if (sms <= 0) return KDA_ERR_CUDA;
  if (f16)
    s = launch_prefill<32, true>(args, m, st);
  else
    s = (int64_t)num_seqs * dims.HV * 4 <= sms ? launch_prefill<32, false>(args, m, st)
                                               : launch_prefill<64, false>(args, m, st);
  record_stage(2, st);
  return s;
}
