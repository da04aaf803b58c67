// kda_logprobs.cu -- log probabilities of given tokens, with the entropy of their
// distributions and their top alternatives.
//
// Of a row's logits x, with m the largest and z = sum exp(x - m):
//   log p_j = x_j - m - log z,   entropy = log z - sum (x - m) exp(x - m) / z.
// One pass over the row: a thread keeps m, z and the sum of the entropy of what it
// has read (rescaled where m grows), and the tile's values stay in registers for
// the search of the alternatives.
//
// Alternatives.  Of 8 warps' threads each takes the largest value of its own; the
// ceil(top / 8)-th largest of those in every warp bounds from below what at least
// top values of the tile reach, so that only values at or above the least of the 8
// bounds (and above every earlier tile's) are candidates: some fifty of the first
// tile's 8192, fewer of each later one.  They go to a list in shared memory, as
// keys that no two entries share: the value's bits in an order of their own, then
// the token's complement, so that among equals the lowest token comes first.  A
// tile with more candidates than the list has room for (rows of one value) is
// searched key by key instead.  At the end a key's rank is the number of larger
// ones.
//
// A row is split over the CTAs of a cluster where there are few rows; rank 0 joins
// what the others leave in its shared memory.
#include <cooperative_groups.h>
#include <float.h>
#include <limits.h>

#include "kda_host.h"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTop = KDA_LOGPROBS_MAX_TOP;
constexpr int kPerThread = 32;  // a tile's values in a thread's registers
constexpr int kTile = kThreads * kPerThread;
constexpr int kList = 2048;     // candidates
constexpr int kMaxCluster = 8;

struct LogprobsArgs {
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  int rows, vocab, top;
  float *logprobs, *entropy;
  int32_t* top_tokens;
  float* top_logprobs;
  int32_t* err_flag;
};

struct Stats {
  float m, z, t;  // largest value, sum exp(x - m), sum (x - m) exp(x - m)
};

// Rank 0's: what the CTAs of a cluster leave for it.
struct Joined {
  unsigned long long keys[kMaxCluster][kMaxTop];
  Stats stats[kMaxCluster];
};

// Whole numbers in the order of the values, -0 as 0; NaN must not come here.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ unsigned long long key_of(float x, int token) {
  return (unsigned long long)ordered(x) << 32 | (uint32_t)~token;
}
constexpr uint32_t kOrderedLowest = 0x00800000u;  // of -FLT_MAX: what is below is -inf, and no alternative

__device__ __forceinline__ Stats join(const Stats& a, const Stats& b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return Stats{m, 0.f, 0.f};
  // differences of -inf are of sums of nothing
  const float da = fmaxf(a.m - m, -1e4f), db = fmaxf(b.m - m, -1e4f), ea = expf(da), eb = expf(db);
  return Stats{m, a.z * ea + b.z * eb, (a.t + a.z * da) * ea + (b.t + b.z * db) * eb};
}

template <int DT>
__device__ __forceinline__ float one(const void* row, int64_t i) {
  if (DT == KDA_DTYPE_F32) return __ldg(static_cast<const float*>(row) + i);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(row) + i);
  return DT == KDA_DTYPE_F16 ? in16_to_float<true>(b) : in16_to_float<false>(b);
}

// A 16-byte piece widened.
template <int DT>
__device__ __forceinline__ void widen(uint4 w, float* x) {
  if (DT == KDA_DTYPE_F32) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  } else {
    const float4 a = in16x4_to_f4<DT == KDA_DTYPE_F16>(make_uint2(w.x, w.y)), b = in16x4_to_f4<DT == KDA_DTYPE_F16>(make_uint2(w.z, w.w));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

struct Lists {
  unsigned long long list[kList], best[kMaxTop], warp_best[kWarps];
  int count;
  uint32_t bound[kWarps];
  Stats stats[kWarps];
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The list's `top` largest keys, in falling order, to `best`, zeros behind them; the
// whole CTA, ends with a barrier.
__device__ __forceinline__ void rank_list(Lists& s, int n, int top) {
  if (threadIdx.x < kMaxTop) s.best[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long mine = s.list[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += s.list[j] > mine;
    if (rank < top) s.best[rank] = mine;
  }
  __syncthreads();
}

template <int DT, bool TOP>
__global__ void __launch_bounds__(kThreads, 3) logprobs_kernel(const LogprobsArgs args) {
  constexpr int kSize = DT == KDA_DTYPE_F32 ? 4 : 2, kEach = 16 / kSize, kPieces = kPerThread / kEach;
  __shared__ Lists s;
  __shared__ Joined joined;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / ranks, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int top = TOP ? args.top : 0;
  const int token = args.tokens[r];
  if (token < 0 || token >= args.vocab) {  // nothing is asked of this row
    if (rank == 0) {
      if (tid == 0) {
        if (token != -1) set_error(args.err_flag, KDA_DEVERR_TOKEN);
        args.logprobs[r] = 0.f;
        if (args.entropy) args.entropy[r] = 0.f;
      }
      if (TOP && tid < top) {
        args.top_tokens[(int64_t)r * top + tid] = -1;
        args.top_logprobs[(int64_t)r * top + tid] = 0.f;
      }
    }
    return;  // the whole cluster
  }
  cluster_arrive();  // rank 0 has started before the others write to it
  const char* row = static_cast<const char*>(args.logits) + (int64_t)r * args.stride * kSize;
  const float x_token = one<DT>(row, token);
  // single entries before the first and behind the last whole 16 bytes, the others in pieces
  const int to_piece = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / kSize;
  const int head = to_piece < args.vocab ? to_piece : args.vocab;
  const int pieces = (args.vocab - head) / kEach, tail = args.vocab - head - pieces * kEach;
  const uint4* body = reinterpret_cast<const uint4*>(row + head * kSize);
  const int tiles = (pieces + kThreads * kPieces - 1) / (kThreads * kPieces);

  if (tid == 0) s.count = 0;
  Stats mine{-INFINITY, 0.f, 0.f};
  uint32_t least = kOrderedLowest;  // what a candidate has to reach
  for (int tile = rank; tile < tiles || tile == 0; tile += ranks) {
    float x[kPerThread + 1];
    int single = -1;  // the token of the single entry
    x[kPerThread] = -INFINITY;
    {
      uint4 w[kPieces] = {};
      const int p0 = tile * kThreads * kPieces + tid;
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if (p0 + j * kThreads < pieces) w[j] = __ldcs(body + p0 + j * kThreads);
      if (tile == 0 && tid < head + tail) {
        single = tid < head ? tid : args.vocab - tail + (tid - head);
        x[kPerThread] = one<DT>(row, single);
      }
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        widen<DT>(w[j], x + j * kEach);
        if (p0 + j * kThreads >= pieces)
#pragma unroll
          for (int e = 0; e < kEach; ++e) x[j * kEach + e] = -INFINITY;
      }
    }
    float big = -INFINITY;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) big = fmaxf(big, x[e]);  // NaN is left out
    if (fmaxf(big, x[kPerThread]) == INFINITY) {  // counts as the largest number
#pragma unroll
      for (int e = 0; e <= kPerThread; ++e) x[e] = x[e] == INFINITY ? FLT_MAX : x[e];
      big = fminf(big, FLT_MAX);
    }
    const float m = fmaxf(mine.m, fmaxf(big, x[kPerThread]));
    if (m > -INFINITY) {
      const float down = fmaxf(mine.m - m, -1e4f), scale = __expf(down);
      float z = mine.z * scale, t = (mine.t + mine.z * down) * scale;
#pragma unroll
      for (int e = 0; e <= kPerThread; ++e) {
        const float d = fmaxf(x[e] - m, -1e4f);  // -inf and NaN: no weight
        const float p = __expf(d);
        z += p;
        t = fmaf(d, p, t);
      }
      mine = Stats{m, z, t};
    }
    if constexpr (TOP) {
      const uint32_t u = ordered(big);
      uint32_t left = u, bound = 0;
      for (int i = 0; i < (top + kWarps - 1) / kWarps; ++i) {
        bound = __reduce_max_sync(0xffffffffu, left);
        if (lane == __ffs(__ballot_sync(0xffffffffu, left == bound)) - 1) left = 0;
      }
      if (lane == 0) s.bound[warp] = bound;
      __syncthreads();
      const int before = s.count;
      bound = s.bound[0];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) bound = min(bound, s.bound[i]);
      const bool full = bound >= least;  // then `top` values reach the bound
      if (full) least = bound;
      __syncthreads();  // everyone has read the count
      auto token_at = [&](int e) {
        return e == kPerThread ? single : head + (tile * kThreads * kPieces + e / kEach * kThreads + tid) * kEach + e % kEach;
      };
      if (max(u, ordered(fmaxf(x[kPerThread], -INFINITY))) >= least) {
        const float bar = unordered(least);
#pragma unroll
        for (int e = 0; e <= kPerThread; ++e)
          if (x[e] >= bar) {
            const int at = atomicAdd(&s.count, 1);
            if (at < kList) s.list[at] = key_of(x[e], token_at(e));
          }
      }
      __syncthreads();
      const int n = s.count;
      if (n > kList) {  // too many at once: the tile's largest keys one by one
        __syncthreads();
        unsigned long long last = ~0ull;
        int found = 0;
        for (; found < top; ++found) {
          unsigned long long k = 0;
#pragma unroll
          for (int e = 0; e <= kPerThread; ++e)
            if (x[e] >= -FLT_MAX) {
              const unsigned long long key = key_of(x[e], token_at(e));
              if (key < last && key > k) k = key;
            }
#pragma unroll
          for (int d = 16; d; d >>= 1) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, k, d);
            k = o > k ? o : k;
          }
          if (lane == 0) s.warp_best[warp] = k;
          __syncthreads();
          k = s.warp_best[0];
          for (int i = 1; i < kWarps; ++i) k = s.warp_best[i] > k ? s.warp_best[i] : k;
          __syncthreads();
          if (k == 0) break;
          if (tid == 0) s.list[before + found] = k;
          last = k;
        }
        if (tid == 0) s.count = before + found;
        __syncthreads();
      }
      if (s.count > kList - 2 * kMaxTop || n > kList) {  // room for the next tile's
        const int have = s.count;
        rank_list(s, have, top);
        if (tid < kMaxTop) s.list[tid] = s.best[tid];
        if (tid == 0) s.count = min(have, top);
        __syncthreads();
      }
      if (full) ++least;  // among equals the lower tokens, which are listed, come first
    }
  }

  // the CTA's part of the row, then the row
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const Stats o{__shfl_xor_sync(0xffffffffu, mine.m, d), __shfl_xor_sync(0xffffffffu, mine.z, d),
                  __shfl_xor_sync(0xffffffffu, mine.t, d)};
    mine = join(mine, o);
  }
  if (lane == 0) s.stats[warp] = mine;
  __syncthreads();
  if constexpr (TOP) rank_list(s, s.count, top);
  cluster_wait();
  Joined* to = cluster.map_shared_rank(&joined, 0);
  if (TOP && tid < kMaxTop) to->keys[rank][tid] = s.best[tid];
  if (tid == 0) {
    Stats all = s.stats[0];
    for (int i = 1; i < kWarps; ++i) all = join(all, s.stats[i]);
    to->stats[rank] = all;
  }
  cluster.sync();
  if (rank != 0) return;
  Stats all = joined.stats[0];
  for (int i = 1; i < ranks; ++i) all = join(all, joined.stats[i]);
  const float log_z = logf(all.z);
  const bool some = all.m > -INFINITY;
  auto log_p = [&](float x) { return some && x >= -FLT_MAX ? (fminf(x, FLT_MAX) - all.m) - log_z : -INFINITY; };
  if (tid == 0) {
    args.logprobs[r] = log_p(x_token);
    if (args.entropy) args.entropy[r] = some ? log_z - all.t / all.z : 0.f;
  }
  if constexpr (TOP) {
    static_assert(kMaxCluster * kMaxTop == kThreads, "a thread per entry");
    const int from = tid / kMaxTop, pos = tid % kMaxTop;
    const unsigned long long key = from < ranks ? joined.keys[from][pos] : 0;
    const int taken = __syncthreads_count(key != 0);
    if (key) {
      int place = pos;
      for (int c = 0; c < ranks; ++c) {
        if (c == from) continue;
        int lo = 0, hi = top;  // entries of that list that are larger
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (joined.keys[c][mid] > key) lo = mid + 1; else hi = mid;
        }
        place += lo;
      }
      if (place < top) {
        args.top_tokens[(int64_t)r * top + place] = (int32_t)~(uint32_t)key;
        args.top_logprobs[(int64_t)r * top + place] = log_p(unordered((uint32_t)(key >> 32)));
      }
    }
    // places that no entry took
    if (tid < top && tid >= taken) {
      args.top_tokens[(int64_t)r * top + tid] = -1;
      args.top_logprobs[(int64_t)r * top + tid] = -INFINITY;
    }
  }
}

template <int DT>
kda_status launch_logprobs(const LogprobsArgs& a, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0) return KDA_ERR_CUDA;
  const int64_t tiles = ((int64_t)a.vocab + kTile - 1) / kTile;
  int ranks = 1;
  while (ranks < kMaxCluster && ranks < tiles && (int64_t)a.rows * ranks < 3 * (int64_t)sms) ranks *= 2;
  if ((int64_t)a.rows * ranks > INT32_MAX) return KDA_ERR_SHAPE;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)ranks, 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.rows * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  record_stage(0, st);
  cudaLaunchKernelEx(&cfg, a.top ? logprobs_kernel<DT, true> : logprobs_kernel<DT, false>, a);
  const kda_status s = launch_status();
  record_stage(1, st);
  record_stage(2, st);
  return s;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_token_logprobs(int logits_dtype, const void* logits, int64_t logits_stride, const int32_t* tokens,
                                         int rows, int vocab, float* logprobs, float* entropy, int top, int32_t* top_tokens,
                                         float* top_logprobs, int32_t* err_flag, void* stream) {
  if (logits_dtype != KDA_DTYPE_F32 && logits_dtype != KDA_DTYPE_BF16 && logits_dtype != KDA_DTYPE_F16) return KDA_ERR_UNSUPPORTED;
  if (rows < 0 || vocab < 1 || top < 0 || logits_stride < vocab) return KDA_ERR_SHAPE;
  if (top > KDA_LOGPROBS_MAX_TOP || vocab > KDA_ACCEPT_MAX_VOCAB) return KDA_ERR_UNSUPPORTED;
  if (rows == 0) return KDA_OK;
  if (!logits || !tokens || !logprobs || (top > 0 && (!top_tokens || !top_logprobs))) return KDA_ERR_NULL_ARG;
  if (reinterpret_cast<uintptr_t>(logits) & (logits_dtype == KDA_DTYPE_F32 ? 3u : 1u)) return KDA_ERR_ALIGNMENT;
  const LogprobsArgs a{logits, logits_stride, tokens, rows, vocab, top, logprobs, entropy, top_tokens, top_logprobs, err_flag};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (logits_dtype) {
    case KDA_DTYPE_F32: return launch_logprobs<KDA_DTYPE_F32>(a, st);
    case KDA_DTYPE_F16: return launch_logprobs<KDA_DTYPE_F16>(a, st);
    default: return launch_logprobs<KDA_DTYPE_BF16>(a, st);
  }
}
