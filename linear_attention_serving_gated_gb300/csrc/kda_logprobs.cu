// kda_logprobs.cu -- log probabilities of given tokens, with the entropy of their
// distributions and their top alternatives.
//
// Of a row's logits x, with m the largest and z = sum exp(x - m) = 1 + r:
//   log p_j = x_j - m - log(1 + r),   entropy = log(1 + r) - sum (x - m) exp(x - m) / (1 + r).
// One pass over the row, in tiles of 16 KiB.  A thread copies its own pieces of a tile
// to shared memory a tile ahead and reads them back itself, so that no barrier stands
// between a load and its use; it keeps m, z and the sum of the entropy of what it has
// read, rescaled where m grows.
//
// Precision.  r is kept without the 1 of the largest value, so that the log probability
// of a token that is all but certain, log(1 + r) with a small r, is as exact as any
// other.  (With 1 + r in FP32 it is off by 2^-23 at best.)  For that a thread sums the
// tile with its largest value apart from the others, and where a warp's r is small the
// entries that its largest value came with are summed once more, without it.  (Counting
// entries equal to m as they come took a sixth more time.)  What is left is 2^-22 of an
// exponential and the rounding of x - m in units of ln 2, 2^-24 |x - m|.
//
// Alternatives.  Of the first tile each thread takes its largest value; the
// ceil(top / 8)-th largest of those in every warp bounds from below what at least top
// values of the tile reach, so that only values at or above the least of the 8 bounds
// are candidates: some fifty of 4096 or 8192.  The pieces that hold some go to a list in
// shared memory as they are.  After 1, 2, 4, 8 .. tiles the CTA takes the candidates out of
// them, as keys that no two entries share (the value's bits in an order of their own, then
// the token's complement, so that among equals the lowest token comes first), ranks these,
// a key's rank being the number of larger ones, and keeps the top largest: the last of them
// is the new bound.  Tiles with more than the lists have room for (rising values, or one
// value) are read again, twice: for a bound from each thread's largest key, and for the
// keys that reach it.
//
// A row is split over the CTAs of a cluster where there are few rows; rank 0 joins
// what the others leave in its shared memory.
//
// 288 rows of 131072 FP32 logits with 20 alternatives take 30 us (5.0 TB/s), without any
// 24.5 (6.1 TB/s): the candidates' way into the lists and out of them.  (Candidates listed
// one by one: 33; with one cut after the first tile: 41; a barrier a tile and rows held in
// registers: 69.)  Six rows of 50257 take 6.7 us, latencies one behind the other.
#include <cooperative_groups.h>
#include <float.h>
#include <limits.h>

#include "kda_host.h"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTop = KDA_LOGPROBS_MAX_TOP;
constexpr int kPieces = 4;      // 16-byte pieces of a tile a thread has
constexpr int kAhead = 2;       // tiles under way
constexpr int kList = 512;      // candidates, and pieces that hold some
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

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
  float m, r, t;  // largest value, sum exp(x - m) - 1, sum (x - m) exp(x - m)
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

// Of the lanes' parts together, in every lane.
__device__ __forceinline__ Stats warp_join(Stats a) {
  float m = a.m;
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (m == -INFINITY) return Stats{m, 0.f, 0.f};
  const float down = fmaxf(a.m - m, -1e4f), e = expf(down);  // (a part of nothing: -inf less m)
  const bool first = __ffs(__ballot_sync(0xffffffffu, a.m == m)) - 1 == (threadIdx.x & 31);
  float r = first ? a.r : (1.f + a.r) * e, t = (a.t + (1.f + a.r) * down) * e;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    r += __shfl_xor_sync(0xffffffffu, r, d);
    t += __shfl_xor_sync(0xffffffffu, t, d);
  }
  return Stats{m, r, t};
}

template <int DT>
__device__ __forceinline__ float one(const void* row, int64_t i) {
  if (DT == KDA_DTYPE_F32) return __ldg(static_cast<const float*>(row) + i);
  const uint16_t b = __ldg(static_cast<const uint16_t*>(row) + i);
  return DT == KDA_DTYPE_F16 ? in16_to_float<true>(b) : in16_to_float<false>(b);
}

template <int DT>
__device__ __forceinline__ float shared_one(const void* from, int i) {
  if (DT == KDA_DTYPE_F32) return static_cast<const float*>(from)[i];
  const uint16_t b = static_cast<const uint16_t*>(from)[i];
  return DT == KDA_DTYPE_F16 ? in16_to_float<true>(b) : in16_to_float<false>(b);
}

struct Lists {
  uint4 ring[kAhead][kPieces][kThreads];
  unsigned long long list[2][kList + kMaxTop], warp_best[kWarps];  // two lists, in turn
  uint4 piece[kList];
  int piece_at[kList];
  int count[2], piece_count;
  uint32_t bound[kWarps];
  Stats stats[kWarps];
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The `top` largest of a list's n keys, in falling order; 0 is none.
__device__ __forceinline__ void rank_keys(const unsigned long long* list, int n, int top, unsigned long long* to) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long mine = list[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += list[j] > mine;
    if (rank < top && mine) to[rank] = mine;
  }
}

__device__ __forceinline__ float no_infinity(float x) { return x == INFINITY ? FLT_MAX : x; }

// 2^x, results below the smallest normal number as zero.
__device__ __forceinline__ float exp2_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two entries of a word (or the two words' one each) widened.
template <int DT>
__device__ __forceinline__ void widen(uint4 w, float2* x) {
  if (DT == KDA_DTYPE_F32) {
    x[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    x[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = DT == KDA_DTYPE_F16 ? __half22float2(*reinterpret_cast<const __half2*>(&u[i]))
                                 : make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  }
}

// The largest of a piece's entries, NaN left out; -inf where there is none.
template <int DT>
__device__ __forceinline__ float piece_max(uint4 w) {
  float2 m;
  if constexpr (DT == KDA_DTYPE_F32) {
    m = make_float2(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  } else if constexpr (DT == KDA_DTYPE_F16) {
    auto h = [](uint32_t u) { return *reinterpret_cast<const __half2*>(&u); };
    m = __half22float2(__hmax2(__hmax2(h(w.x), h(w.y)), __hmax2(h(w.z), h(w.w))));
  } else {
    auto b = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
    m = __bfloat1622float2(__hmax2(__hmax2(b(w.x), b(w.y)), __hmax2(b(w.z), b(w.w))));
  }
  return fmaxf(-INFINITY, fmaxf(m.x, m.y));
}

template <int DT, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobsArgs args) {
  constexpr int kSize = DT == KDA_DTYPE_F32 ? 4 : 2, kEach = 16 / kSize;
  __shared__ __align__(16) Lists s;
  __shared__ Joined joined;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = blockIdx.x / ranks, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int top = TOP ? args.top : 0;
  const char* row = static_cast<const char*>(args.logits) + (int64_t)r * args.stride * kSize;
  // single entries before the first and behind the last whole 16 bytes, the others in pieces
  const int to_piece = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / kSize;
  const int head = to_piece < args.vocab ? to_piece : args.vocab;
  const int pieces = (args.vocab - head) / kEach, tail = args.vocab - head - pieces * kEach;
  const uint4* body = reinterpret_cast<const uint4*>(row + head * kSize);
  const int tiles = (pieces + kThreads * kPieces - 1) / (kThreads * kPieces);
  auto piece_of = [&](int tile, int j) { return (tile * kPieces + j) * kThreads + tid; };
  auto whole = [&](int tile) { return (tile + 1) * (kPieces * kThreads) <= pieces; };
  // the single entries in front with the first tile, those behind with rank 0's last one,
  // so that a CTA's tokens come in order (but within a tile)
  auto single_of = [&](int tile) {
    if (rank != 0) return -1;
    if (tile + ranks >= tiles && tid >= 32 && tid < 32 + tail) return args.vocab - tail + tid - 32;
    return tile == 0 && tid < head ? tid : -1;
  };
  auto fetch = [&](int tile, int slot) {  // (one group for every tile, of nothing behind the last)
    if (whole(tile)) {
      const uint4* from = body + piece_of(tile, 0);
#pragma unroll
      for (int j = 0; j < kPieces; ++j) cp_async16(&s.ring[slot][j][tid], from + j * kThreads);
    } else if (tile < tiles) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if (piece_of(tile, j) < pieces) cp_async16(&s.ring[slot][j][tid], body + piece_of(tile, j));
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(rank + i * ranks, i);
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
    cp_async_wait_all();
    return;  // the whole cluster
  }
  cluster_arrive();  // rank 0 has started before the others write to it
  const float x_token = one<DT>(row, token);

  if (tid == 0) s.count[0] = s.piece_count = 0;
  if (TOP) __syncthreads();
  float top_x = -INFINITY;  // the largest value so far,
  int top_tile = 0;         // the tile that it came with,
  float top_z = 0.f;        // that tile's part of z
  float z = 0.f;            // and the others'
  float2 t = make_float2(0.f, 0.f);
  uint32_t least = kOrderedLowest;  // what a candidate has to reach
  int slot = 0, batch = rank, seen = 0;  // the first tile since the last look at the list; tiles so far
  int cur = 0;                           // the list in use
  for (int tile = rank; tile < tiles || tile == 0; tile += ranks) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    uint4 w[kPieces];
    // a missing piece holds -inf
    constexpr uint32_t kNone = DT == KDA_DTYPE_F32 ? 0xff800000u : DT == KDA_DTYPE_F16 ? 0xfc00fc00u : 0xff80ff80u;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) w[j] = s.ring[slot][j][tid];
    fetch(tile + kAhead * ranks, slot);
    slot ^= 1;
    if (!whole(tile)) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if (piece_of(tile, j) >= pieces) w[j] = make_uint4(kNone, kNone, kNone, kNone);
    }
    const int single = single_of(tile);
    const float x_single = single >= 0 ? one<DT>(row, single) : -INFINITY;
    float2 x[kEach / 2];
    float big = -INFINITY, piece_big[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      piece_big[j] = piece_max<DT>(w[j]);
      big = fmaxf(big, piece_big[j]);
    }
    // +inf counts as the largest number
    const float m = fmaxf(top_x, fminf(fmaxf(big, x_single), FLT_MAX));
    const bool fresh = m > top_x;
    if (fresh) {
      const float down = fmaxf(top_x - m, -1e4f), scale = exp2_(down * kLog2e);
      z += top_z;
      t = make_float2(fmaf(z, down, t.x) * scale, t.y * scale);
      z *= scale;
      top_x = m;
      top_tile = tile;
    }
    if (m > -INFINITY) {
      const float2 minus = make_float2(-m, -m);
      float2 sum = make_float2(0.f, 0.f);
      auto add = [&](float2 v) {
        const float2 d = add2(v, minus);
        const float2 c = make_float2(fmaxf(d.x, -1e4f), fmaxf(d.y, -1e4f));  // -inf and NaN: no weight
        const float2 y = mul2(c, make_float2(kLog2e, kLog2e));
        const float2 p = make_float2(exp2_(y.x), exp2_(y.y));
        sum = add2(sum, p);
        t = fma2(c, p, t);
      };
      if (big < INFINITY) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          widen<DT>(w[j], x);
#pragma unroll
          for (int e = 0; e < kEach / 2; ++e) add(x[e]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          widen<DT>(w[j], x);
#pragma unroll
          for (int e = 0; e < kEach / 2; ++e) add(make_float2(no_infinity(x[e].x), no_infinity(x[e].y)));
        }
      }
      if (single >= 0) add(make_float2(no_infinity(x_single), -INFINITY));
      const float part = sum.x + sum.y;
      if (fresh) top_z = part; else z += part;
    }
    if constexpr (TOP) {
      auto each = [&](uint4 w, int piece, auto&& f) {  // a piece's entries
        widen<DT>(w, x);
#pragma unroll
        for (int e = 0; e < kEach / 2; ++e) {
          f(x[e].x, head + piece * kEach + 2 * e);
          f(x[e].y, head + piece * kEach + 2 * e + 1);
        }
      };
      const uint32_t u = ordered(fminf(big, FLT_MAX));
      if (tile == rank) {
        uint32_t left = u, bound = 0;
        for (int i = 0; i < (top + kWarps - 1) / kWarps; ++i) {
          bound = __reduce_max_sync(0xffffffffu, left);
          if (lane == __ffs(__ballot_sync(0xffffffffu, left == bound)) - 1) left = 0;
        }
        if (lane == 0) s.bound[warp] = bound;
        __syncthreads();
        bound = s.bound[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) bound = min(bound, s.bound[i]);
        least = max(least, bound);
      }
      const float bar = unordered(least);
      auto list = [&](float v, int at) {
        if (v >= bar) {
          const int i = atomicAdd(&s.count[cur], 1);
          if (i < kList) s.list[cur][i] = key_of(no_infinity(v), at);
        }
      };
      if (u >= least) {
        int at = 0;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) at += piece_big[j] >= bar;
        at = atomicAdd(&s.piece_count, at);
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          if (piece_big[j] >= bar && at < kList) {
            s.piece[at] = w[j];
            s.piece_at[at++] = piece_of(tile, j);
          }
        }
      }
      if (single >= 0) list(x_single, single);
      ++seen;
      if ((seen & (seen - 1)) == 0 || tile + ranks >= tiles) {
        const int from = batch;
        batch = tile + ranks;
        unsigned long long *keys = s.list[cur], *next = s.list[cur ^ 1];
        __syncthreads();
        int n = s.piece_count;
        if (n <= kList) {
          for (int i = tid; i < n * kEach; i += kThreads)  // an entry a thread
            list(shared_one<DT>(s.piece, i), head + s.piece_at[i / kEach] * kEach + i % kEach);
          __syncthreads();
          n = s.count[cur];
        }
        if (n > kList) {  // too many: the tiles since are read again
          __syncthreads();  // all have read how many pieces there are, which is counted anew below
          // What is listed of them, whose tokens are higher than earlier ones', is not the lot.
          const uint32_t first = from == 0 ? 0 : head + from * (kPieces * kThreads * kEach);
          const int have = min(s.count[cur], kList);
          auto again = [&](auto&& f) {  // their keys
            auto entry = [&](float v, int at) {
              if (v >= -FLT_MAX) f(key_of(no_infinity(v), at));
            };
#pragma unroll 1
            for (int t = from; t <= tile; t += ranks)
#pragma unroll 1
              for (int j = 0; j < kPieces; ++j)
                if (piece_of(t, j) < pieces) each(__ldg(body + piece_of(t, j)), piece_of(t, j), entry);
            // the single entries: of the first tile, or of the last one
            if (rank == 0 && from == 0 && tid < head) entry(one<DT>(row, tid), tid);
            if (single >= head) entry(x_single, single);
          };
          // The top-th largest of the threads' largest keys bounds them.
          unsigned long long *largest = reinterpret_cast<unsigned long long*>(s.piece), *some = largest + kThreads;
          constexpr int kSome = (int)(sizeof(s.piece) / 8) - kThreads;
          unsigned long long mine = 0;
          again([&](unsigned long long key) { mine = key > mine ? key : mine; });
          largest[tid] = mine;
          if (tid < kMaxTop) next[tid] = 0;
          if (tid == 0) s.piece_count = 0, s.warp_best[0] = 0;
          __syncthreads();
          int larger = 0;
          for (int i = 0; i < kThreads; ++i) larger += largest[i] > mine;
          if (mine && larger == top - 1) s.warp_best[0] = mine;
          __syncthreads();
          const unsigned long long bound = s.warp_best[0];
          auto take = [&](unsigned long long key) {
            const int i = atomicAdd(&s.piece_count, 1);
            if (i < kSome) some[i] = key;
          };
          again([&](unsigned long long key) {
            if (key >= bound) take(key);
          });
          for (int i = tid; i < have; i += kThreads)
            if (~(uint32_t)keys[i] < first) take(keys[i]);
          __syncthreads();
          n = s.piece_count;
          if (n <= kSome) {
            rank_keys(some, n, top, next);
          } else {  // (a few threads have them all) the largest key, and again
            for (int i = tid; i < kList; i += kThreads)
              if (i >= have || ~(uint32_t)keys[i] >= first) keys[i] = 0;
            unsigned long long last = ~0ull;
            int found = 0;
            for (; found < top; ++found) {
              unsigned long long k = 0;
              again([&](unsigned long long key) {
                if (key < last && key > k) k = key;
              });
#pragma unroll
              for (int d = 16; d; d >>= 1) {
                const unsigned long long o = __shfl_xor_sync(0xffffffffu, k, d);
                k = o > k ? o : k;
              }
              __syncthreads();
              if (lane == 0) s.warp_best[warp] = k;
              __syncthreads();
              k = s.warp_best[0];
              for (int i = 1; i < kWarps; ++i) k = s.warp_best[i] > k ? s.warp_best[i] : k;
              if (k == 0) break;
              if (tid == 0) keys[kList + found] = k;
              last = k;
            }
            __syncthreads();
            rank_keys(keys, kList + found, top, next);
          }
          __syncthreads();
          n = __syncthreads_count(tid < top && next[tid] != 0);
        } else {
          rank_keys(keys, n, top, next);
        }
        cur ^= 1;
        if (tid == 0) s.count[cur] = min(n, top), s.piece_count = 0;
        __syncthreads();
        if (n >= top) least = max(least, (uint32_t)(next[top - 1] >> 32) + 1);
      }
    }
  }
  cp_async_wait_all();

  // the warp's part of the row, then the CTA's, then the row
  {
    float m = top_x;
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const int most = __ffs(__ballot_sync(0xffffffffu, top_x == m)) - 1;
    const float down = fmaxf(top_x - m, -1e4f), e = expf(down);
    float r = lane == most ? z : (z + top_z) * e, all_t = (t.x + t.y + (z + top_z) * down) * e;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      r += __shfl_xor_sync(0xffffffffu, r, d);
      all_t += __shfl_xor_sync(0xffffffffu, all_t, d);
    }
    float mine = __shfl_sync(0xffffffffu, top_z - 1.f, most);
    if (m == -INFINITY) {
      mine = r = all_t = 0.f;
    } else if (r + mine < 0.25f) {  // a lane for each piece, one for the single entry
      const int tile = __shfl_sync(0xffffffffu, top_tile, most), single = __shfl_sync(0xffffffffu, single_of(top_tile), most);
      const int piece = piece_of(tile, lane) - lane + most;
      mine = 0.f;
      auto add = [&](float v) {
        const float d = no_infinity(v) - m;
        if (d != 0.f) mine += expf(fmaxf(d, -1e4f));
      };
      if (lane < kPieces && piece < pieces) {
        float2 x[kEach / 2];
        widen<DT>(__ldg(body + piece), x);
#pragma unroll
        for (int i = 0; i < kEach / 2; ++i) add(x[i].x), add(x[i].y);
      } else if (lane == kPieces && single >= 0) {
        add(one<DT>(row, single));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
    }
    if (lane == 0) s.stats[warp] = Stats{m, r + mine, all_t};
  }
  __syncthreads();
  cluster_wait();
  Joined* to = cluster.map_shared_rank(&joined, 0);
  // (the last tile's look at the list; a CTA of the single entries' share has no tile)
  if (TOP && tid < kMaxTop) to->keys[rank][tid] = tid < s.count[cur] ? s.list[cur][tid] : 0;
  if (warp == 0) {
    const Stats all = warp_join(lane < kWarps ? s.stats[lane] : Stats{-INFINITY, 0.f, 0.f});
    if (lane == 0) to->stats[rank] = all;
  }
  cluster.sync();
  if (rank != 0) return;
  const Stats all = warp_join(lane < ranks ? joined.stats[lane] : Stats{-INFINITY, 0.f, 0.f});
  const float log_z = log1pf(all.r);
  const bool some = all.m > -INFINITY;
  auto log_p = [&](float x) { return some && x >= -FLT_MAX ? (fminf(x, FLT_MAX) - all.m) - log_z : -INFINITY; };
  if (tid == 0) {
    args.logprobs[r] = log_p(x_token);
    if (args.entropy) args.entropy[r] = some ? log_z - all.t / (1.f + all.r) : 0.f;
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
  constexpr int kTile = kThreads * kPieces * (DT == KDA_DTYPE_F32 ? 4 : 8);
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
