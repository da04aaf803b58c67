// kda_pool.cu -- pages of a state pool: copy, free, compact, fork.
//
// A page is one slot's record in every layer (1 MiB a layer at 16 heads of
// 128 x 128 FP32).  The moved bytes bound these calls: each page is read once
// and written once.  Bookkeeping is a byte per slot and a table row per
// request, all on the device, so that a call can be captured and replayed.
//
// Which page goes where is a question of ranks: the k-th free slot, the k-th
// used one at or above the new top.  A CTA answers it from a bitmap of the
// used slots in shared memory (one bit a slot) with a running count per
// 32-bit word: a binary search over the words, then a bit scan.  A pool of
// 240 slots is 8 words, so every CTA of a copy builds its own instead of
// waiting for a plan in memory.
#include <limits.h>

#include <atomic>

#include "kda_host.h"

namespace kda {
namespace {

constexpr int kMaxSlots = 1 << 19;  // (bitmap + counts) 4 bytes + 4 bytes per 32 slots: 128 KiB
constexpr int kThreads = 256;
constexpr int kVec = 4;  // 16-byte pieces a thread has in flight
constexpr int kPartBytes = kThreads * kVec * 16;

// Bitmap of the used slots and the number of used slots before each word.
struct UsedMap {
  uint32_t* bits;
  int* before;  // [words + 1]
  int words, slots;

  __device__ int total() const { return before[words]; }
  __device__ int used_below(int s) const {
    const int w = s >> 5;
    return w >= words ? total() : before[w] + __popc(bits[w] & ((1u << (s & 31)) - 1u));
  }
  // the slot of the k-th (from 0) used / free slot; it must exist
  template <bool FREE>
  __device__ int select(int k) const {
    int lo = 0, hi = words - 1;  // the last word with at most k before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      const int b = FREE ? mid * 32 - before[mid] : before[mid];
      if (b <= k) lo = mid; else hi = mid - 1;
    }
    k -= FREE ? lo * 32 - before[lo] : before[lo];
    uint32_t m = FREE ? ~bits[lo] : bits[lo];
    for (; k > 0; --k) m &= m - 1;
    return lo * 32 + __ffs(m) - 1;
  }
};

// Built by the whole CTA (blockDim.x a multiple of 32); ends with a barrier.
__device__ UsedMap build_map(const uint8_t* used, int slots, uint32_t* smem) {
  __shared__ int warp_sum[32];
  __shared__ int carry_s;
  UsedMap m;
  m.words = (slots + 31) / 32;
  m.slots = slots;
  m.bits = smem;
  m.before = reinterpret_cast<int*>(smem + m.words);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockDim.x;
  if (tid == 0) carry_s = 0;
  __syncthreads();
  for (int w0 = 0; w0 < m.words; w0 += n) {
    const int w = w0 + tid;
    uint32_t b = 0;
    if (w < m.words) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // four slots a load
        const int s = w * 32 + j * 4;
        uint32_t x = 0;
        if (s + 3 < slots)
          x = __ldcg(reinterpret_cast<const uint32_t*>(used + s));
        else
          for (int e = 0; s + e < slots; ++e) x |= (uint32_t)__ldcg(used + s + e) << (8 * e);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (x >> (8 * e) & 0xffu) b |= 1u << (j * 4 + e);
      }
      m.bits[w] = b;
    }
    const int c = __popc(b);
    int x = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int base = carry_s;
    for (int i = 0; i < warp; ++i) base += warp_sum[i];
    if (w < m.words) m.before[w] = base + x - c;
    __syncthreads();
    if (tid == n - 1) carry_s = base + x;
    __syncthreads();
  }
  if (tid == 0) m.before[m.words] = carry_s;
  __syncthreads();
  return m;
}

size_t map_bytes(int slots) { return ((size_t)(slots + 31) / 32) * 8 + 8; }

// One CTA's part of a page copy: kPartBytes of one layer, every thread's loads
// in flight before its first store.  src < 0 writes zeros.
__device__ __forceinline__ void copy_part(const kda_pages& pg, int64_t layer, int64_t part, int src, int dst) {
  const int64_t n16 = pg.page_bytes / 16;
  char* base = static_cast<char*>(pg.base) + layer * pg.layer_stride;
  const uint4* s = reinterpret_cast<const uint4*>(base + (int64_t)(src < 0 ? 0 : src) * pg.page_bytes);
  uint4* d = reinterpret_cast<uint4*>(base + (int64_t)dst * pg.page_bytes);
  const int64_t i0 = part * (kPartBytes / 16) + threadIdx.x;
  uint4 v[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const int64_t i = i0 + e * kThreads;
    v[e] = src >= 0 && i < n16 ? __ldcs(s + i) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const int64_t i = i0 + e * kThreads;
    if (i < n16) d[i] = v[e];
  }
}

__global__ void __launch_bounds__(kThreads) page_copy_kernel(const kda_pages pg, const int32_t* src, const int32_t* dst,
                                                             int n, int parts, int32_t* err_flag) {
  const int64_t per_pair = (int64_t)parts * pg.layers;
  const int i = (int)(blockIdx.x / per_pair);
  const int64_t rest = blockIdx.x % per_pair;
  const int s = src[i], d = dst[i];
  if (s == -1 || d == -1) return;
  bool bad = s < 0 || d < 0 || s >= pg.slots || d >= pg.slots;
  for (int j = threadIdx.x; j < n && !bad; j += kThreads)
    bad |= j != i && src[j] != -1 && dst[j] != -1 && (dst[j] == d || src[j] == d);
  if (__syncthreads_or(bad)) {
    if (rest == 0 && threadIdx.x == 0) set_error(err_flag, KDA_DEVERR_PAGE);
    return;
  }
  copy_part(pg, rest / parts, rest % parts, s, d);
}

__global__ void __launch_bounds__(kThreads) page_free_kernel(uint8_t* used, int slots, int32_t* table, int table_rows,
                                                             const int32_t* rows, int n, int32_t* err_flag) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  const int row = rows[i];
  if (row == -1) return;
  if (row < 0 || row >= table_rows) {
    set_error(err_flag, KDA_DEVERR_PAGE);
    return;
  }
  const int s = atomicExch(table + row, -1);  // a row listed twice frees its page once
  if (s == -1) return;
  if (s < 0 || s >= slots) {
    set_error(err_flag, KDA_DEVERR_PAGE);
    return;
  }
  const uint32_t m = 0xffu << (8 * (s & 3));
  const uint32_t old = atomicAnd(reinterpret_cast<uint32_t*>(used) + (s >> 2), ~m);
  if (!(old & m)) set_error(err_flag, KDA_DEVERR_PAGE);
}

// Compaction, first kernel: the moves.  CTAs walk over (move, layer, part).
__global__ void __launch_bounds__(kThreads) compact_copy_kernel(const kda_pages pg, const uint8_t* used, int parts) {
  extern __shared__ uint32_t map_smem[];
  grid_dependency_launch();
  const UsedMap m = build_map(used, pg.slots, map_smem);
  const int count = m.total(), below = m.used_below(count);
  const int64_t per_move = (int64_t)parts * pg.layers, total = (int64_t)(count - below) * per_move;
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    const int k = (int)(t / per_move);
    const int64_t rest = t % per_move;
    copy_part(pg, rest / parts, rest % parts, m.select<false>(below + k), m.select<true>(k));
  }
}

// Second kernel: table, used and count, once the first has read them.
__global__ void __launch_bounds__(1024) compact_update_kernel(uint8_t* used, int slots, int32_t* table, int table_rows,
                                                              int32_t* count_out, int32_t* err_flag) {
  extern __shared__ uint32_t map_smem[];
  const UsedMap m = build_map(used, slots, map_smem);
  const int count = m.total(), below = m.used_below(count);
  grid_dependency_wait();
  for (int r = threadIdx.x; r < table_rows; r += blockDim.x) {
    const int s = table[r];
    if (s == -1) continue;
    if (s < 0 || s >= slots || !(m.bits[s >> 5] >> (s & 31) & 1u))
      set_error(err_flag, KDA_DEVERR_PAGE);
    else if (s >= count)
      table[r] = m.select<true>(m.used_below(s) - below);
  }
  for (int s = threadIdx.x; s < slots; s += blockDim.x) used[s] = s < count;
  if (threadIdx.x == 0) *count_out = count;
}

// Whether table row `par` holds a page that was in use before the call (a page
// given out by this call is not in the map).
__device__ __forceinline__ bool has_page(const UsedMap& m, const int32_t* table, int par) {
  const int s = __ldcg(table + par);
  return s >= 0 && s < m.slots && (m.bits[s >> 5] >> (s & 31) & 1u);
}

// Fork, first kernel: which row gets which page.  Rows without a page are
// claimed with the marker INT_MIN + i, the lowest i that lists the row winning,
// so that a row listed twice is served once; claims are then counted in order.
// (A row of another value below -1 holds no slot there is: refused.)
__global__ void __launch_bounds__(1024) fork_assign_kernel(uint8_t* used, int slots, int32_t* table, int table_rows,
                                                           const int32_t* parents, const int32_t* rows, int n,
                                                           int32_t* children, int32_t* err_flag) {
  extern __shared__ uint32_t map_smem[];
  __shared__ int warp_sum[32];
  grid_dependency_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const UsedMap m = build_map(used, slots, map_smem);
  const int free_pages = slots - m.total();
  for (int i = tid; i < n; i += blockDim.x) {
    const int row = rows[i];
    if (row < 0 || row >= table_rows) {
      if (row != -1) set_error(err_flag, KDA_DEVERR_PAGE);
      continue;
    }
    const int mine = INT_MIN + i;
    int old = table[row];
    while (old == -1 || (old > mine && old < INT_MIN + n)) {
      const int seen = atomicCAS(table + row, old, mine);
      if (seen == old) break;
      old = seen;
    }
  }
  __syncthreads();
  int given = 0;
  for (int i0 = 0; i0 < n; i0 += blockDim.x) {
    const int i = i0 + tid;
    const int row = i < n ? rows[i] : -1;
    const bool named = row >= 0 && row < table_rows;
    const bool mine = named && __ldcg(table + row) == INT_MIN + i;
    bool win = mine;
    if (mine) {
      const int par = parents[i];
      win = par == -1 || (par >= 0 && par < table_rows && has_page(m, table, par));
    }
    if (named && !win) set_error(err_flag, KDA_DEVERR_PAGE);  // listed before, holds a page or none there is, or no parent
    const unsigned b = __ballot_sync(0xffffffffu, win);
    if (lane == 0) warp_sum[warp] = __popc(b);
    __syncthreads();  // and every marker of this round has been read
    int k = given + __popc(b & ((1u << lane) - 1u)), all = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
      if (w < warp) k += warp_sum[w];
      all += warp_sum[w];
    }
    int s = -1;
    if (mine) {
      if (win && k < free_pages) {
        s = m.select<true>(k);
        used[s] = 1;
      } else if (win) {
        set_error(err_flag, KDA_DEVERR_POOL_FULL);
      }
      table[row] = s;
    }
    if (i < n) children[i] = s;
    given += all;
    __syncthreads();
  }
}

// Second kernel: the copies.  An entry that got a page has a parent whose page
// was in use before the call, which the first kernel has not touched.
__global__ void __launch_bounds__(kThreads) fork_copy_kernel(const kda_pages pg, const int32_t* table,
                                                             const int32_t* parents, const int32_t* children, int parts) {
  const int64_t per_pair = (int64_t)parts * pg.layers;
  const int i = (int)(blockIdx.x / per_pair);
  const int64_t rest = blockIdx.x % per_pair;
  const int par = parents[i];
  grid_dependency_wait();
  const int d = children[i];
  if (d >= 0) copy_part(pg, rest / parts, rest % parts, par >= 0 ? table[par] : -1, d);
}

kda_status check_pages(const kda_pages& p) {
  if (!p.base) return KDA_ERR_NULL_ARG;
  if (p.slots < 1 || p.layers < 1 || p.page_bytes < 16 || p.layer_stride < 0) return KDA_ERR_SHAPE;
  if (p.slots > kMaxSlots) return KDA_ERR_UNSUPPORTED;
  if (!aligned16(p.base) || p.page_bytes % 16 != 0 || p.layer_stride % 16 != 0) return KDA_ERR_ALIGNMENT;
  if (p.page_bytes > INT64_MAX / kMaxSlots || (p.layers > 1 && p.layer_stride < p.page_bytes * p.slots)) return KDA_ERR_SHAPE;
  return KDA_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The shared-memory limits of the kernels that hold a map of `bytes`.  Without
// one a kernel gets 48 KiB, its own arrays (under 1 KiB) among them.  Set for the
// largest map, in the first call on a device that needs more: a later one may be
// under capture.
bool allow_map(size_t bytes) {
  static std::atomic<uint64_t> ready{0};
  if (bytes + 1024 <= 48 * 1024) return true;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (ready.load(std::memory_order_relaxed) >> dev & 1u) return true;
  auto allow = [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)map_bytes(kMaxSlots)) == cudaSuccess;
  };
  if (!allow(compact_copy_kernel) || !allow(compact_update_kernel) || !allow(fork_assign_kernel)) return false;
  ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  return true;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_pool_copy(kda_pages pages, const int32_t* src, const int32_t* dst, int n, int32_t* err_flag,
                                    void* stream) {
  kda_status s = check_pages(pages);
  if (s != KDA_OK) return s;
  if (n < 0) return KDA_ERR_SHAPE;
  if (n == 0) return KDA_OK;
  if (!src || !dst) return KDA_ERR_NULL_ARG;
  const int64_t parts = (pages.page_bytes + kPartBytes - 1) / kPartBytes;
  if (parts > INT32_MAX || parts * pages.layers > INT32_MAX / n) return KDA_ERR_SHAPE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  record_stage(0, st);
  page_copy_kernel<<<(unsigned)(parts * pages.layers * n), kThreads, 0, st>>>(pages, src, dst, n, (int)parts, err_flag);
  s = launch_status();
  record_stage(1, st);
  record_stage(2, st);
  return s;
}

extern "C" kda_status kda_pool_free(uint8_t* used, int slots, int32_t* table, int table_rows, const int32_t* rows, int n,
                                    int32_t* err_flag, void* stream) {
  if (slots < 1 || table_rows < 0 || n < 0) return KDA_ERR_SHAPE;
  if (n == 0) return KDA_OK;
  if (!used || !table || !rows) return KDA_ERR_NULL_ARG;
  if (!aligned4(used)) return KDA_ERR_ALIGNMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  record_stage(0, st);
  page_free_kernel<<<(n + kThreads - 1) / kThreads, kThreads, 0, st>>>(used, slots, table, table_rows, rows, n, err_flag);
  const kda_status s = launch_status();
  record_stage(1, st);
  record_stage(2, st);
  return s;
}

extern "C" kda_status kda_pool_compact(kda_pages pages, uint8_t* used, int32_t* table, int table_rows, int32_t* count,
                                       int32_t* err_flag, void* stream) {
  kda_status s = check_pages(pages);
  if (s != KDA_OK) return s;
  if (table_rows < 0) return KDA_ERR_SHAPE;
  if (!used || !count || (table_rows > 0 && !table)) return KDA_ERR_NULL_ARG;
  if (!aligned4(used)) return KDA_ERR_ALIGNMENT;
  const int64_t parts = (pages.page_bytes + kPartBytes - 1) / kPartBytes;
  if (parts > INT32_MAX) return KDA_ERR_SHAPE;
  const int sms = sm_count();
  if (sms <= 0) return KDA_ERR_CUDA;
  const size_t smem = map_bytes(pages.slots);
  if (!allow_map(smem)) return KDA_ERR_CUDA;
  // at most half of the slots move (a move fills a hole)
  const double most = (double)parts * pages.layers * (pages.slots / 2 + 1);
  const unsigned grid = (unsigned)(most < 8.0 * sms ? most : 8.0 * sms);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  record_stage(0, st);
  compact_copy_kernel<<<grid, kThreads, smem, st>>>(pages, used, (int)parts);
  record_stage(1, st);
  s = launch_status();
  if (s != KDA_OK) return s;
  s = launch_dependent(compact_update_kernel, 1, 1024, smem, !stage_between(), st, used, pages.slots, table, table_rows, count,
                       err_flag);
  record_stage(2, st);
  return s;
}

extern "C" kda_status kda_pool_fork(kda_pages pages, uint8_t* used, int32_t* table, int table_rows,
                                    const int32_t* parents, const int32_t* rows, int n, int32_t* children,
                                    int32_t* err_flag, void* stream) {
  kda_status s = check_pages(pages);
  if (s != KDA_OK) return s;
  if (table_rows < 0 || n < 0) return KDA_ERR_SHAPE;
  if (n == 0) return KDA_OK;
  if (!used || !table || !parents || !rows || !children) return KDA_ERR_NULL_ARG;
  if (!aligned4(used)) return KDA_ERR_ALIGNMENT;
  const int64_t parts = (pages.page_bytes + kPartBytes - 1) / kPartBytes;
  if (parts > INT32_MAX || parts * pages.layers > INT32_MAX / n) return KDA_ERR_SHAPE;
  const size_t smem = map_bytes(pages.slots);
  if (!allow_map(smem)) return KDA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  record_stage(0, st);
  fork_assign_kernel<<<1, 1024, smem, st>>>(used, pages.slots, table, table_rows, parents, rows, n, children,
                                                err_flag);
  record_stage(1, st);
  s = launch_status();
  if (s != KDA_OK) return s;
  s = launch_dependent(fork_copy_kernel, (unsigned)(parts * pages.layers * n), kThreads, 0, !stage_between(), st, pages,
                       static_cast<const int32_t*>(table), parents, static_cast<const int32_t*>(children), (int)parts);
  record_stage(2, st);
  return s;
}
