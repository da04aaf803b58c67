// kda_tc.cuh -- sm_100-family tensor-core, TMEM, mbarrier and bulk-copy
// primitives (inline PTX) used by the prefill kernels.
//
// Operand layout, but where a function says otherwise (TF32 tiles, operands
// stored MN-major): BF16 or FP16, K-major, 128-byte swizzle.  A tile
// of R rows and K columns (K a multiple of 64) is stored as K/64 "atom
// columns"; atom column a holds columns [64a, 64a+64) of every row, one
// 128-byte line per row, rows consecutive, so 8 rows form a 1024-byte swizzle
// atom.  Inside a line the 16-byte chunk index is XORed with (row % 8).
// Every atom column starts on a 1024-byte boundary.
#pragma once

#include <stdint.h>

namespace kda {
namespace tc {

// ---------------------------------------------------------------------------
// Shared-memory addressing

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Byte offset of element (row, col) inside a swizzled K-major BF16 tile with
// `rows` rows.
__device__ __forceinline__ uint32_t sw128_offset(int row, int col, int rows) {
  const int atom = col >> 6, cc = col & 63;
  const uint32_t chunk = static_cast<uint32_t>((cc >> 3) ^ (row & 7));
  return static_cast<uint32_t>(atom * rows * 128 + row * 128) + (chunk << 4) +
         static_cast<uint32_t>((cc & 7) << 1);
}

// As sw128_offset for a 32-bit (TF32) tile: 32 elements per 128-byte line,
// atom column a holds columns [32a, 32a+32).
__device__ __forceinline__ uint32_t sw128_offset_f32(int row, int col, int rows) {
  const int atom = col >> 5, cc = col & 31;
  const uint32_t chunk = static_cast<uint32_t>((cc >> 2) ^ (row & 7));
  return static_cast<uint32_t>(atom * rows * 128 + row * 128) + (chunk << 4) +
         static_cast<uint32_t>((cc & 3) << 2);
}

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups
// 1024 bytes apart (stride byte offset), leading byte offset unused for this
// layout (encoded as 1), descriptor version 1, base offset 0.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;                 // LBO (unused) = 16 B
  d |= static_cast<uint64_t>(1024u >> 4) << 32;         // SBO = 1024 B
  d |= static_cast<uint64_t>(1u) << 46;                 // version
  d |= static_cast<uint64_t>(2u) << 61;                 // SWIZZLE_128B
  return d;
}

// As sw128_desc for an operand stored MN-major: 128-byte lines of 64
// consecutive rows (M or N) of one k, lines of consecutive k 128 bytes apart.
// Eight k form a 1024-byte swizzle atom (stride byte offset); the next 64
// rows follow `rows64_bytes` further on (leading byte offset).
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t smem_addr, uint32_t rows64_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((rows64_bytes >> 4) & 0x3FFFu) << 16;  // LBO
  d |= static_cast<uint64_t>(1024u >> 4) << 32;                     // SBO
  d |= static_cast<uint64_t>(1u) << 46;                             // version
  d |= static_cast<uint64_t>(2u) << 61;                             // SWIZZLE_128B
  return d;
}

// The same for an operand of 32 or 16 rows: lines of 64 or 32 bytes, eight of
// which form an atom, swizzled in 16-byte pieces within 64 or 32 bytes.
template <int ROWS>
__device__ __forceinline__ uint64_t sw_desc_mn(uint32_t smem_addr) {
  static_assert(ROWS == 32 || ROWS == 16, "rows");
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((ROWS * 16) >> 4) << 32;         // SBO
  d |= static_cast<uint64_t>(1u) << 46;                       // version
  d |= static_cast<uint64_t>(ROWS == 32 ? 4u : 6u) << 61;     // SWIZZLE_64B, SWIZZLE_32B
  return d;
}

// Operand majors of an instruction descriptor: set for an MN-major A or B.
constexpr uint32_t kIdescMnA = 1u << 15, kIdescMnB = 1u << 16;

// Instruction descriptor of kind::f16 with BF16 A/B, FP32 accumulator,
// both operands K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N) {
  return (1u << 4)                                   // D format F32
         | (1u << 7)                                 // A format BF16
         | (1u << 10)                                // B format BF16
         | (static_cast<uint32_t>(N >> 3) << 17)     // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);    // M / 16
}

// The same with FP16 A/B (format 0).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return idesc_bf16_f32(M, N) & ~((1u << 7) | (1u << 10));
}

// Instruction descriptor of kind::tf32: TF32 A/B, FP32 accumulator, both
// operands K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_tf32_f32(int M, int N) {
  return (1u << 4)                                   // D format F32
         | (2u << 7)                                 // A format TF32
         | (2u << 10)                                // B format TF32
         | (static_cast<uint32_t>(N >> 3) << 17)     // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);    // M / 16
}

// ---------------------------------------------------------------------------
// mbarrier

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait: returns false if the phase did not complete within the limit.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, uint32_t limit = 1u << 22) {
  for (uint32_t i = 0; i < limit; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

// ---------------------------------------------------------------------------
// Bulk copy global -> shared (no tensor map), completion on an mbarrier.
// dst, src 16-byte aligned, bytes a multiple of 16.

__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Bulk copy shared -> global (no tensor map), tracked by this thread's bulk
// groups.  src, dst 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// Bulk prefetch of global memory into L2 (no shared memory involved).  src
// 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// Waits until every committed bulk store of this thread has finished reading
// shared memory (the source may then be overwritten).
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Fences

// Generic-proxy shared-memory writes -> visible to the async proxy (MMA, bulk copy).
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// ---------------------------------------------------------------------------
// TMEM allocation (one full warp executes these)

__device__ __forceinline__ void tmem_alloc(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(smem_dst)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// ---------------------------------------------------------------------------
// MMA: D[tmem] (+)= A[smem] * B[smem]^T, issued by one thread.

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// As mma_bf16 for TF32 operands (K = 8 per instruction, 32 bytes of each row).
__device__ __forceinline__ void mma_tf32(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// Arrive on an mbarrier once all MMAs issued so far by this thread complete.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// ---------------------------------------------------------------------------
// TMEM -> registers: warp w reads lanes [32*(w%4), +32), 16 consecutive
// 32-bit columns starting at `col`; thread i gets lane 32*(w%4)+i.

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// As tmem_ld16 without the wait: the registers are valid after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// As tmem_ld16, 8 columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Split an FP32 value into a BF16 pair hi + lo with hi = RN(x), lo = RN(x - hi).
__device__ __forceinline__ void split_bf16(float x, uint16_t& hi, uint16_t& lo) {
  const __nv_bfloat16 h = __float2bfloat16_rn(x);
  hi = __bfloat16_as_ushort(h);
  lo = __bfloat16_as_ushort(__float2bfloat16_rn(x - __bfloat162float(h)));
}

// FP32 -> TF32 rounded to nearest, ties away from zero, low 13 bits zero, so
// that the tensor core's use of the top 19 bits is exact.  Done on the bit
// pattern (sign-magnitude: adding half a TF32 unit to the magnitude and
// dropping the low bits rounds half away from zero; a carry into the exponent
// gives the next binade) with two integer operations; finite inputs only.
__device__ __forceinline__ uint32_t tf32_rna(float x) {
  return (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
}

// Four consecutive values of row `row`, columns [col, col+4) (col a multiple
// of 4), rounded to TF32 into a swizzled K-major 32-bit tile of `rows` rows.
__device__ __forceinline__ void st_tf32x4(uint8_t* tile, int row, int col, int rows, float4 x) {
  *reinterpret_cast<uint4*>(tile + sw128_offset_f32(row, col, rows)) =
      make_uint4(tf32_rna(x.x), tf32_rna(x.y), tf32_rna(x.z), tf32_rna(x.w));
}

}  // namespace tc
}  // namespace kda
