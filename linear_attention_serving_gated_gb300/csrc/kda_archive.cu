// kda_archive.cu -- pages of a state pool kept in 8 or 4 bits, and read back.
//
// A group of values x (128 in 8 bits, 32 in 4) shares an FP32 scale:
//   scale = max|x| / top,  code = x / scale rounded to nearest, ties to even,
// top = 127 or 7; read back, a value is code * scale.  Bound by HBM: 4 bytes read
// and 1.03 (0.625) written a value, and the other way round.  A warp takes rows of
// 128 values, four a lane, eight rows with all their loads in flight; the largest
// magnitude of a row is one warp reduction of bit patterns, that of a group of 32
// three exchanges.  70 pages of 4 MiB stored and read back in 8 bits: 123 us, 6.0 TB/s,
// 88% of a copy's rate; codes by conversions 139 us, and loads behind the check of the
// pairs 148.
#include "kda_host.h"

namespace kda {
namespace {

constexpr int kThreads = 256, kRowsPerWarp = 8, kRow = 128;
constexpr int kPartRows = kThreads / 32 * kRowsPerWarp;  // rows of a CTA: 32 KB of a page

struct ArchiveArgs {
  kda_pages pages;
  uint8_t* codes;
  float* scales;
  int slots;
  const int32_t *src, *dst;
  int n;
  int64_t rows;  // of 128 values, of a page in one layer
  int parts;     // CTAs of such a page
  int32_t* err_flag;
};

// What a CTA works on.  Its loads start as soon as its own pair is known to be in range;
// whether another pair has the same destination is found out while they are under way.
struct Work {
  int pair, src, dst;
  int64_t layer, row0;  // this warp's first row
  bool in_range;
};
__device__ __forceinline__ Work find_work(const ArchiveArgs& a, int src_slots, int dst_slots) {
  Work w;
  const int64_t per_pair = (int64_t)a.parts * a.pages.layers;
  w.pair = (int)(blockIdx.x / per_pair);
  const int64_t rest = blockIdx.x % per_pair;
  w.src = a.src[w.pair];
  w.dst = a.dst[w.pair];
  w.in_range = w.src >= 0 && w.dst >= 0 && w.src < src_slots && w.dst < dst_slots;
  w.layer = rest / a.parts;
  w.row0 = rest % a.parts * kPartRows + (int64_t)(threadIdx.x >> 5) * kRowsPerWarp;
  return w;
}
// Whether the pair is one to copy; the whole CTA, a barrier.
__device__ __forceinline__ bool accept(const ArchiveArgs& a, const Work& w) {
  if (w.src == -1 || w.dst == -1) return false;
  bool bad = !w.in_range;
  for (int j = threadIdx.x; j < a.n && !bad; j += kThreads) bad |= j != w.pair && a.src[j] != -1 && a.dst[j] == w.dst;
  if (!__syncthreads_or(bad)) return true;
  if (blockIdx.x % ((int64_t)a.parts * a.pages.layers) == 0 && threadIdx.x == 0) set_error(a.err_flag, KDA_DEVERR_PAGE);
  return false;
}

// The code of x, settled where x times 1 / scale may have fallen on the wrong side of a
// half: the remainder x - c scale is exact (a whole number of the operands' last places,
// below the scale).
__device__ __forceinline__ int code_of(float x, float scale, float inv, float top) {
  float c = rintf(x * inv);
  const float r = fmaf(-c, scale, x), twice = 2.f * fabsf(r);
  const bool odd = (__float2int_rn(c) & 1) != 0;
  if (twice > scale || (twice == scale && odd)) c += copysignf(1.f, r);
  return __float2int_rn(fminf(fmaxf(c, -top), top));
}

template <int BITS>
__global__ void __launch_bounds__(kThreads, 4) archive_store_kernel(const ArchiveArgs a) {
  constexpr float kTop = BITS == 8 ? 127.f : 7.f;
  const Work w = find_work(a, a.pages.slots, a.slots);
  const int lane = threadIdx.x & 31;
  const float4* page = reinterpret_cast<const float4*>(static_cast<const char*>(a.pages.base) + w.layer * a.pages.layer_stride +
                                                       (int64_t)w.src * a.pages.page_bytes);
  const int64_t to = ((int64_t)w.dst * a.pages.layers + w.layer) * a.rows;  // the archive's row of row 0
  float4 x[kRowsPerWarp];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i)
    x[i] = w.in_range && w.row0 + i < a.rows ? __ldcs(page + (w.row0 + i) * (kRow / 4) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
  if (!accept(a, w)) return;
  float mine = 0.f;  // the scale that this lane stores
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const uint32_t b0 = __float_as_uint(x[i].x) & 0x7fffffffu, b1 = __float_as_uint(x[i].y) & 0x7fffffffu,
                   b2 = __float_as_uint(x[i].z) & 0x7fffffffu, b3 = __float_as_uint(x[i].w) & 0x7fffffffu;
    uint32_t m = max(max(b0, b1), max(b2, b3));
    if (BITS == 8) {
      m = __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    }
    // a group that holds an infinity or a NaN reads back as NaN
    const bool finite = m < 0x7f800000u;
    float scale = finite ? __fdiv_rn(__uint_as_float(m), kTop) : __uint_as_float(0x7fffffffu);
    // 127 times the scale of the largest FP32 number is past it; the one below is not
    if (BITS == 8 && scale > 0x1.020406p121f) scale = 0x1.020406p121f;
    int c[4] = {0, 0, 0, 0};
    const float v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    if (finite && scale >= 1e-37f) {
      // x / scale rounded by adding 1.5 * 2^23, whose low bits are then the code; a
      // remainder that is not below half a scale is one in a million, and settled exactly
      const float inv = __frcp_rn(scale), half = 0.5f * scale;
      bool close = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y = fmaf(v[e], inv, 12582912.f);
        close |= fabsf(fmaf(12582912.f - y, scale, v[e])) >= half;
        c[e] = __float_as_int(y) - 0x4b400000;
      }
      if (close)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = code_of(v[e], scale, inv, kTop);
    } else if (finite && scale > 0.f) {  // 1 / scale may be out of range; such quotients have few places and are exact enough to round
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = __double2int_rn(fmin(fmax((double)v[e] / (double)scale, -(double)kTop), (double)kTop));
    }
    const int64_t row = to + w.row0 + i;
    if (w.row0 + i < a.rows) {
      if (BITS == 8)
        reinterpret_cast<uint32_t*>(a.codes)[row * (kRow / 4) + lane] =
            __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
      else
        reinterpret_cast<uint16_t*>(a.codes)[row * (kRow / 4) + lane] =
            (uint16_t)((c[0] & 15) | (c[1] & 15) << 4 | (c[2] & 15) << 8 | (c[3] & 15) << 12);
    }
    if (BITS == 8) {
      if (lane == i) mine = scale;
    } else {
      const float s = __shfl_sync(0xffffffffu, scale, 8 * (lane & 3));
      if (lane >> 2 == i) mine = s;
    }
  }
  if (BITS == 8) {
    if (lane < kRowsPerWarp && w.row0 + lane < a.rows) a.scales[to + w.row0 + lane] = mine;
  } else {
    if (w.row0 + (lane >> 2) < a.rows) a.scales[(to + w.row0) * 4 + lane] = mine;
  }
}

template <int BITS>
__global__ void __launch_bounds__(kThreads, 5) archive_load_kernel(const ArchiveArgs a) {
  const Work w = find_work(a, a.slots, a.pages.slots);
  const int lane = threadIdx.x & 31;
  float4* page = reinterpret_cast<float4*>(static_cast<char*>(a.pages.base) + w.layer * a.pages.layer_stride +
                                           (int64_t)w.dst * a.pages.page_bytes);
  const int64_t from = ((int64_t)w.src * a.pages.layers + w.layer) * a.rows;
  uint32_t c[kRowsPerWarp];
  float s[kRowsPerWarp];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int64_t row = from + w.row0 + i;
    c[i] = 0;
    s[i] = 0.f;
    if (w.in_range && w.row0 + i < a.rows) {
      if (BITS == 8) {
        c[i] = __ldcs(reinterpret_cast<const uint32_t*>(a.codes) + row * (kRow / 4) + lane);
        s[i] = __ldcs(a.scales + row);
      } else {
        c[i] = __ldcs(reinterpret_cast<const uint16_t*>(a.codes) + row * (kRow / 4) + lane);
        s[i] = __ldcs(a.scales + row * 4 + (lane >> 3));
      }
    }
  }
  if (!accept(a, w)) return;
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    if (w.row0 + i >= a.rows) continue;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // the code plus 128 (or 8) as the low bits of 2^23 (conversions run at a quarter of this rate)
      const uint32_t u = BITS == 8 ? __byte_perm(c[i] ^ 0x80808080u, 0x4b000000u, 0x7650 | e)
                                   : (((c[i] ^ 0x8888u) >> (4 * e)) & 15u) | 0x4b000000u;
      v[e] = (__uint_as_float(u) - (BITS == 8 ? 8388736.f : 8388616.f)) * s[i];
    }
    page[(w.row0 + i) * (kRow / 4) + lane] = make_float4(v[0], v[1], v[2], v[3]);
  }
}

kda_status run_archive(const kda_pages& pg, const kda_archive& ar, const int32_t* src, const int32_t* dst, int n,
                       int32_t* err_flag, void* stream, bool store) {
  if (ar.bits != 8 && ar.bits != 4) return KDA_ERR_UNSUPPORTED;
  if (!pg.base || !ar.codes || !ar.scales) return KDA_ERR_NULL_ARG;
  if (pg.slots < 1 || pg.layers < 1 || pg.page_bytes < 1 || pg.layer_stride < 0 || ar.slots < 1 || n < 0) return KDA_ERR_SHAPE;
  if (!aligned16(pg.base) || pg.layer_stride % 16 != 0 || !aligned16(ar.codes) || !aligned16(ar.scales)) return KDA_ERR_ALIGNMENT;
  if (pg.page_bytes % (kRow * 4) != 0) return KDA_ERR_UNSUPPORTED;
  if (pg.page_bytes > INT64_MAX / pg.slots || (pg.layers > 1 && pg.layer_stride < pg.page_bytes * pg.slots)) return KDA_ERR_SHAPE;
  if (n == 0) return KDA_OK;
  if (!src || !dst) return KDA_ERR_NULL_ARG;
  ArchiveArgs a{pg, static_cast<uint8_t*>(ar.codes), ar.scales, ar.slots, src, dst, n, pg.page_bytes / (kRow * 4), 0, err_flag};
  const int64_t parts = (a.rows + kPartRows - 1) / kPartRows;
  if (parts > INT32_MAX || parts * pg.layers > INT32_MAX / n) return KDA_ERR_SHAPE;
  a.parts = (int)parts;
  const unsigned grid = (unsigned)(parts * pg.layers * n);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  record_stage(0, st);
  if (store)
    (ar.bits == 8 ? archive_store_kernel<8> : archive_store_kernel<4>)<<<grid, kThreads, 0, st>>>(a);
  else
    (ar.bits == 8 ? archive_load_kernel<8> : archive_load_kernel<4>)<<<grid, kThreads, 0, st>>>(a);
  const kda_status s = launch_status();
  record_stage(1, st);
  record_stage(2, st);
  return s;
}

}  // namespace
}  // namespace kda

extern "C" kda_status kda_pool_store(kda_pages pages, kda_archive archive, const int32_t* src, const int32_t* dst, int n,
                                     int32_t* err_flag, void* stream) {
  return kda::run_archive(pages, archive, src, dst, n, err_flag, stream, true);
}

extern "C" kda_status kda_pool_load(kda_pages pages, kda_archive archive, const int32_t* src, const int32_t* dst, int n,
                                    int32_t* err_flag, void* stream) {
  return kda::run_archive(pages, archive, src, dst, n, err_flag, stream, false);
}
