// kda_accept.cu -- verification of drafted tokens against the target's
// probabilities, chain and tree, and the draw of the token behind them.
//
// Chain: drafted token i stands while u_i q_i < p_i.  With a the last row that
// stands, the next token comes from max(p - q, 0) of target row a and draft
// row a (the draft that fell), or from p behind the last row.  Tree: the walk
// of include/kda.h.  The next token is the lowest j whose running sum of
// weights passes u times their whole.
//
// The answer is a whole number, so it must not depend on how sums are split.
// A chain's accept tests are exact: the product of two FP32 numbers fits FP64; a
// tree's are FP64.  Sums of weights are FP32 pairs (sum, error) whose error part
// takes what each addition and each difference p - q rounds off (two-sum), and so
// is u times the whole: within 2^-40 of the whole for up to 2^20 entries (see Pair).
// FP64, at 1/64 of FP32's rate here, is left to the accept tests.
//
// One cluster per request: every CTA repeats the walk (a few gathered loads,
// whose latency is the same for one CTA as for all), its warps sum blocks of 256
// weights and store one pair per block in the first CTA's shared memory.  The
// first CTA scans the block sums, and its warps go through the block that holds
// the border.  A row is read once, 32 bytes a lane and block.  Bound by latency for
// a few requests: 1 x 6 of 32000 FP32 entries 6.2 us, of which the walk 1.5, the
// sums 2, their exchange and scan 1.5, the border 1.3; 16 trees of 6, 50257, 9.2.
// 48 x 6 of 131072, 50 MB of p and q, 15.6 us, 3.2 TB/s or 48% of a copy's rate.
#include <cooperative_groups.h>

#include <atomic>

#include "kda_host.h"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kAccThreads = 256, kAccWarps = kAccThreads / 32;
constexpr int kBlock = 256;      // weights per block sum, 8 a lane
constexpr int kMaxBlocks = 1024;  // longer rows take larger blocks
constexpr int kRing = 4;          // groups of 256 weights a warp has under way to shared memory
// 16-byte pieces of a group a lane takes, of p and of q
template <int DT>
constexpr int kPieces = DT == KDA_DTYPE_F32 ? 2 : 1;
template <int DT>
constexpr int kRingBytes = kRing * 2 * kPieces<DT> * 16 * kAccThreads;

struct AcceptArgs {
  const void* target;
  int64_t target_stride;
  const void* draft;
  int64_t draft_stride;
  const int32_t* tokens;
  const int32_t* parent;
  const float* uniforms;
  const int32_t* lengths;
  int T, vocab;
  int32_t *accepted, *path, *next_token;
  int32_t* err_flag;
};

template <int DT>
__device__ __forceinline__ float prob_at(const void* p, int64_t i) {
  float x;
  if constexpr (DT == KDA_DTYPE_F32)
    x = __ldg(static_cast<const float*>(p) + i);
  else
    x = in16_to_float<DT == KDA_DTYPE_F16>(__ldg(static_cast<const uint16_t*>(p) + i));
  // NaN, negative and infinite entries count as zero
  return x > 0.f && x < __int_as_float(0x7f800000) ? x : 0.f;
}

// The row a request draws from: weights max(p - q, 0), p without the tokens
// that fell (skip), or p alone.
struct Row {
  const void* p;
  const void* q;     // nullptr: no draft row
  int64_t p0, q0;    // element offsets of the rows
  const int* skip;   // tokens that fell
  int n_skip;
};

__device__ __forceinline__ float valid(float x) {  // NaN, negative and infinite entries count as zero
  x = fmaxf(x, 0.f);
  return x < __int_as_float(0x7f800000) ? x : 0.f;
}

// Eight entries of a row: j, j + step, ..; zeros past the end.  VEC: step is 1 and
// j a multiple of 8 of a row that starts on 16 bytes.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* base, int64_t row0, int j, int step, int V, float (&x)[8]) {
  if (VEC && j + 8 <= V) {
    if constexpr (DT == KDA_DTYPE_F32) {
      const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(base) + row0 + j);
      const float4 a = __ldg(s), b = __ldg(s + 1);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + row0 + j));
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = in16_to_float<DT == KDA_DTYPE_F16>((uint16_t)(e & 1 ? ww[e / 2] >> 16 : ww[e / 2] & 0xffffu));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = j + e * step;
      x[e] = 0.f;
      if (k < V) {
        if constexpr (DT == KDA_DTYPE_F32)
          x[e] = __ldg(static_cast<const float*>(base) + row0 + k);
        else
          x[e] = in16_to_float<DT == KDA_DTYPE_F16>(__ldg(static_cast<const uint16_t*>(base) + row0 + k));
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = valid(x[e]);
}

// max(p - q, 0), exactly w + err (p and q valid; where p > q the difference's
// rounding is (p - w) - q).
__device__ __forceinline__ void difference(float p, float q, float& w, float& err) {
  const float d = p - q;
  err = d > 0.f ? (p - d) - q : 0.f;
  w = fmaxf(d, 0.f);
}

// Eight weights as w + err.
template <int DT, bool VEC>
__device__ __forceinline__ void weights8(const Row& row, int j, int step, int V, float (&w)[8], float (&err)[8]) {
  load8<DT, VEC>(row.p, row.p0, j, step, V, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) err[e] = 0.f;
  if (row.q) {
    float q[8];
    load8<DT, VEC>(row.q, row.q0, j, step, V, q);
#pragma unroll
    for (int e = 0; e < 8; ++e) difference(w[e], q[e], w[e], err[e]);
  } else {
    for (int k = 0; k < row.n_skip; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (row.skip[k] == j + e * step) w[e] = 0.f;
  }
}

// A sum as s + c, s rounded and c what that leaves.  The k-th addition in a row
// loses k 2^-48 of the sum at most, as c may have gathered k roundings of s by then:
// sums of many terms move c into s every few of them (tidy).  For up to 2^20 entries
// 16 additions a lane and some 20 of their sums come to 2^-40; a block of 2^28 adds
// 4 a group, 1024 groups: 2^-34.
struct Pair {
  float s, c;
};
__device__ __forceinline__ Pair tidy(Pair x) {
  const float t = x.s + x.c;
  return {t, x.c - (t - x.s)};
}
__device__ __forceinline__ bool operator>(Pair a, Pair b) {  // where it is close, a.s - b.s is exact
  return (a.s - b.s) + (a.c - b.c) > 0.f;
}
__device__ __forceinline__ Pair times(float u, Pair x) {
  const float h = u * x.s;
  return {h, fmaf(u, x.s, -h) + u * x.c};
}
// Where the whole is below 2^-60, u times it would lose bits below FP32's smallest
// number: such rows are drawn from with all weights 2^64 times as large (exact).
__device__ __forceinline__ float lift_of(Pair whole) { return whole.s < 0x1p-60f ? 0x1p64f : 1.f; }
__device__ __forceinline__ Pair operator*(float lift, Pair x) { return {lift * x.s, lift * x.c}; }
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const float t = a.s + b.s, z = t - a.s;
  return {t, a.c + (((a.s - (t - z)) + (b.s - z)) + b.c)};
}
__device__ __forceinline__ Pair shfl(Pair x, int lane) {
  return {__shfl_sync(0xffffffffu, x.s, lane), __shfl_sync(0xffffffffu, x.c, lane)};
}
// Two sums side by side in packed FP32 arithmetic.
struct Pair2 {
  float2 s, c;
  __device__ void add(float2 x, float2 err) {
    const float2 neg = make_float2(-1.f, -1.f);
    const float2 t = add2(s, x), z = fma2(s, neg, t);
    const float2 a = fma2(fma2(z, neg, t), neg, s), b = fma2(z, neg, x);  // s - (t - z), x - z
    c = add2(c, add2(add2(a, b), err));
    s = t;
  }
  __device__ void tidy() {
    const float2 neg = make_float2(-1.f, -1.f);
    const float2 t = add2(s, c);
    c = fma2(fma2(s, neg, t), neg, c);
    s = t;
  }
  __device__ Pair joined() const { return Pair{s.x, c.x} + Pair{s.y, c.y}; }
};
template <int WIDTH>
__device__ __forceinline__ Pair scan(Pair x, int lane) {  // inclusive, over WIDTH lanes
#pragma unroll
  for (int d = 1; d < WIDTH; d <<= 1) {
    const Pair y{__shfl_up_sync(0xffffffffu, x.s, d), __shfl_up_sync(0xffffffffu, x.c, d)};
    if (lane >= d) x = y + x;
  }
  return x;
}

// Sums of a CTA's warps, and what each found.
struct Found {
  Pair sum[kAccWarps];
  int over[kAccWarps], last[kAccWarps];
};

// The lowest j in [lo, hi) with weight whose running sum from `before` exceeds
// `goal` (both `lift` times as large); where rounding leaves none, the last j with weight; -1 where none has
// any.  All warps, 256 weights each at a time; lo a multiple of 8.
template <int DT, bool VEC>
__device__ int find_in(const Row& row, int lo, int hi, float lift, Pair before, Pair goal, Found& f, int warp, int lane) {
  int last = -1;
  for (int base = lo; base < hi; base += kAccWarps * kBlock) {
    const int j0 = base + warp * kBlock;
    float w[8], err[8];
    weights8<DT, VEC>(row, j0 < hi ? j0 + 8 * lane : hi, 1, hi, w, err);
    Pair sum{0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] *= lift;
      err[e] *= lift;
      sum = sum + Pair{w[e], err[e]};
    }
    const Pair in_warp = scan<32>(sum, lane);
    if (lane == 31) f.sum[warp] = in_warp;
    __syncthreads();
    Pair up_to = before;  // this warp's weights
#pragma unroll
    for (int g = 0; g < kAccWarps; ++g) {
      if (g == warp) up_to = before;
      before = before + f.sum[g];
    }
    before = tidy(before);
    const Pair cum = up_to + in_warp;
    const unsigned some = __ballot_sync(0xffffffffu, sum.s > 0.f);
    const unsigned over = __ballot_sync(0xffffffffu, sum.s > 0.f && cum > goal);
    int mine_last = -1;
    if (some) {
      // lane L's eight weights, one each for the first lanes
      const int L = over ? __ffs(over) - 1 : 31 - __clz(some);
      const Pair up = shfl(cum, (L + 31) & 31), start = L > 0 ? up : up_to;
      Pair mine{0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const Pair x = shfl(Pair{w[e], err[e]}, L);
        if (lane == e) mine = x;
      }
      const Pair run = start + scan<8>(mine, lane);
      const unsigned pos = __ballot_sync(0xffffffffu, lane < 8 && mine.s > 0.f);
      const unsigned hit = __ballot_sync(0xffffffffu, lane < 8 && mine.s > 0.f && run > goal);
      mine_last = j0 + 8 * L + (hit ? __ffs(hit) - 1 : 31 - __clz(pos));
    }
    if (lane == 0) {
      f.over[warp] = over ? mine_last : -1;
      f.last[warp] = mine_last;
    }
    __syncthreads();
#pragma unroll
    for (int g = kAccWarps - 1; g >= 0; --g)
      if (f.last[g] >= 0) {
        last = f.last[g];
        break;
      }
#pragma unroll
    for (int g = 0; g < kAccWarps; ++g)
      if (f.over[g] >= 0) return f.over[g];
  }
  return last;
}

template <int DT, bool TREE, bool VEC>
__global__ void __launch_bounds__(kAccThreads, 3) accept_kernel(const AcceptArgs args) {
  cg::cluster_group cluster = cg::this_cluster();
  auto started = cluster.barrier_arrive();
  const int rank = cluster.block_rank(), parts = cluster.num_blocks();
  const int r = blockIdx.x / parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = args.T, V = args.vocab;
  __shared__ float p_tok[TREE ? KDA_ACCEPT_MAX_T : 1], u_s[TREE ? KDA_ACCEPT_MAX_T : 1];
  __shared__ int tok_s[TREE ? KDA_ACCEPT_MAX_T : 1], par_s[TREE ? KDA_ACCEPT_MAX_T : 1];
  __shared__ int skip_s[TREE ? KDA_ACCEPT_MAX_T : 1];
  __shared__ Pair sums[kMaxBlocks], warp_sum[kAccWarps], pick_before;
  __shared__ int first_fall, cur_s, n_skip_s, pick, lowest, highest;
  __shared__ Found found;
  extern __shared__ __align__(16) uint8_t ring_smem[];

  const int64_t r0 = (int64_t)r * T;
  const float u_draw = args.uniforms[r0];
  int n = args.lengths ? args.lengths[r] : T;
  const bool report = rank == 0 && tid == 0;
  if (n < 0 || n > T) {
    if (report) set_error(args.err_flag, KDA_DEVERR_SEQLENS);
    n = 0;
  }
  if (tid == 0) {
    first_fall = n;
    n_skip_s = 0;
    lowest = kAccThreads;
    highest = -1;
  }
  if constexpr (TREE) {
    bool bad = false;
    for (int i = tid; i < n; i += kAccThreads) {
      const int p = args.parent[r0 + i];
      par_s[i] = p;
      bad |= i == 0 ? p != -1 : (p < 0 || p >= i);
    }
    if (__syncthreads_or(bad)) {
      if (report) set_error(args.err_flag, KDA_DEVERR_PARENT);
      n = 0;
    }
  } else {
    __syncthreads();
  }
  // the drafted tokens' probabilities and, for a chain, their tests
  for (int i = 1 + tid; i < T; i += kAccThreads) {
    const int tok = args.tokens[r0 + i];
    const float u = args.uniforms[r0 + i];
    if (i >= n) continue;
    const bool in = tok >= 0 && tok < V;
    if (!in && rank == 0) set_error(args.err_flag, KDA_DEVERR_TOKEN);
    const int up = TREE ? par_s[i] : i - 1;
    const float p = in ? prob_at<DT>(args.target, (r0 + up) * args.target_stride + tok) : 0.f;
    if constexpr (TREE) {
      p_tok[i] = p;
      tok_s[i] = tok;
      u_s[i] = u;
    } else {
      const float q = !in ? 0.f
                          : args.draft ? prob_at<DT>(args.draft, ((int64_t)r * (T - 1) + i - 1) * args.draft_stride + tok)
                                       : 1.f;
      if (!((double)u * (double)q < (double)p)) atomicMin(&first_fall, i);
    }
  }
  __syncthreads();
  if constexpr (TREE) {
    if (tid == 0) {
      // children follow their parents, so one pass over the nodes is the walk
      int cur = 0, n_skip = 0, depth = 0;
      double left = 1.0;
      if (report && n > 0) args.path[r0] = 0;
      for (int i = 1; i < n; ++i) {
        if (par_s[i] != cur) continue;
        double p = p_tok[i];
        for (int s = 0; s < n_skip; ++s)
          if (skip_s[s] == tok_s[i]) p = 0.0;
        if ((double)u_s[i] * left < p) {
          cur = i;
          n_skip = 0;
          left = 1.0;
          ++depth;
          if (report) args.path[r0 + depth] = i;
        } else {
          left -= p;
          skip_s[n_skip++] = tok_s[i];
        }
      }
      n_skip_s = n_skip;
      if (report)
        for (int i = n > 0 ? depth + 1 : 0; i < T; ++i) args.path[r0 + i] = -1;
      cur_s = cur;
    }
    __syncthreads();
  }
  const int cur = TREE ? cur_s : first_fall - 1;
  if (report) args.accepted[r] = n > 0 ? cur : -1;
  if (n == 0) {  // the same for every CTA of the cluster
    cluster.barrier_wait(std::move(started));
    if (report) args.next_token[r] = -1;
    return;
  }
  Row row{args.target, nullptr, (r0 + cur) * args.target_stride, 0, skip_s, n_skip_s};
  if (!TREE && cur + 1 < n) {
    if (args.draft) {
      row.q = args.draft;
      row.q0 = ((int64_t)r * (T - 1) + cur) * args.draft_stride;
    } else {
      row.skip = args.tokens + r0 + cur + 1;
      row.n_skip = 1;
    }
  }
  // block sums, blocks dealt out to the cluster's warps
  // A block sum takes a warp as many instructions as 128 weights do: rows that
  // are long enough take blocks of 1024.
  const int least = (V + kBlock * kMaxBlocks - 1) / (kBlock * kMaxBlocks);
  const int groups = V >= 1024 * parts * kAccWarps && least < 4 ? 4 : least, size = groups * kBlock;
  const int blocks = (V + size - 1) / size;
  const int stride = parts * kAccWarps, b0 = rank * kAccWarps + warp;
  bool waited = false;
  auto store = [&](Pair sum, int b) {
#pragma unroll
    for (int m = 16; m; m >>= 1)
      sum = sum + Pair{__shfl_xor_sync(0xffffffffu, sum.s, m), __shfl_xor_sync(0xffffffffu, sum.c, m)};
    if (!waited) {  // every CTA of the cluster has started: its shared memory may be written
      cluster.barrier_wait(std::move(started));
      waited = true;
    }
    if (lane == 0) *cluster.map_shared_rank(&sums[b], 0) = sum;
  };
  if constexpr (VEC) {
    // Groups of 256 weights pass through a ring in shared memory, kRing of them
    // under way.  A lane reads only the pieces it copied, so its own wait is all
    // the synchronisation there is.
    constexpr int kP = kPieces<DT>, kEl = 8 / kP;  // entries per 16-byte piece
    uint4* ring = reinterpret_cast<uint4*>(ring_smem) + warp * (kRing * 2 * kP * 32) + lane;
    const int mine = b0 < blocks ? (blocks - b0 + stride - 1) / stride * groups : 0;  // groups of this warp
    const bool has_q = row.q != nullptr;
    constexpr int kBytes = DT == KDA_DTYPE_F32 ? 4 : 2;
    const char* p_row = static_cast<const char*>(row.p) + row.p0 * kBytes;
    const char* q_row = has_q ? static_cast<const char*>(row.q) + row.q0 * kBytes : p_row;
    int next = 0, next_j = b0 * size + lane * kEl, next_g = 0;  // the group requested next
    auto request = [&] {
      if (next < mine) {
        uint4* dst = ring + (next % kRing) * (2 * kP * 32);
#pragma unroll
        for (int x = 0; x < kP; ++x) {
          const int j = next_j + x * 32 * kEl, left = (V - j) * kBytes;
          const int bytes = left >= 16 ? 16 : left > 0 ? left : 0;  // zeros past the end
          const int64_t at = bytes ? (int64_t)j * kBytes : 0;
          cp_async16_zfill(dst + x * 32, p_row + at, bytes);
          if (has_q) cp_async16_zfill(dst + (kP + x) * 32, q_row + at, bytes);
        }
        ++next;
        next_j += kBlock;
        if (++next_g == groups) {
          next_g = 0;
          next_j += (stride - 1) * size;
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) request();
    auto value = [&](const uint4& w, int e) {
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      if constexpr (DT == KDA_DTYPE_F32) return __uint_as_float(ww[e]);
      return in16_to_float<DT == KDA_DTYPE_F16>((uint16_t)(e & 1 ? ww[e / 2 % 4] >> 16 : ww[e / 2 % 4] & 0xffffu));
    };
    int k = 0;
    for (int b = b0; b < blocks; b += stride) {
      // Without a look at infinities: a p of them ends up in the sum, the largest
      // q is kept, and a block that has met one is summed again, entry by entry.
      Pair2 sum{make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      float q_max = 0.f;
      for (int g = 0; g < groups; ++g, ++k) {
        request();
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        const uint4* src = ring + (k % kRing) * (2 * kP * 32);
#pragma unroll
        for (int x = 0; x < kP; ++x) {
          const uint4 wp = src[x * 32];
          if (has_q) {
            const uint4 wq = src[(kP + x) * 32];
#pragma unroll
            for (int e = 0; e < kEl; e += 2) {
              const float2 neg = make_float2(-1.f, -1.f);
              const float2 p = make_float2(fmaxf(value(wp, e), 0.f), fmaxf(value(wp, e + 1), 0.f));
              const float2 q = make_float2(fmaxf(value(wq, e), 0.f), fmaxf(value(wq, e + 1), 0.f));
              q_max = fmaxf(q_max, fmaxf(q.x, q.y));
              const float2 d = fma2(q, neg, p), r = fma2(q, neg, fma2(d, neg, p));  // difference()
              sum.add(make_float2(fmaxf(d.x, 0.f), fmaxf(d.y, 0.f)),
                      make_float2(d.x > 0.f ? r.x : 0.f, d.y > 0.f ? r.y : 0.f));
            }
          } else {
            float w[kEl];
#pragma unroll
            for (int e = 0; e < kEl; ++e) w[e] = fmaxf(value(wp, e), 0.f);
            const int j = b * size + g * kBlock + x * 32 * kEl + lane * kEl;
            for (int s = 0; s < row.n_skip; ++s)
#pragma unroll
              for (int e = 0; e < kEl; ++e)
                if (row.skip[s] == j + e) w[e] = 0.f;
#pragma unroll
            for (int e = 0; e < kEl; e += 2) sum.add(make_float2(w[e], w[e + 1]), make_float2(0.f, 0.f));
          }
        }
        sum.tidy();
      }
      Pair total = sum.joined();
      const float inf = __int_as_float(0x7f800000);
      if (__any_sync(0xffffffffu, !(total.s < inf) || !(q_max < inf))) {
        total = Pair{0.f, 0.f};
        for (int j = b * size + 8 * lane; j < b * size + size; j += kBlock) {
          float w[8], err[8];
          weights8<DT, true>(row, j < V ? j : V, 1, V, w, err);
#pragma unroll
          for (int e = 0; e < 8; ++e) total = total + Pair{w[e], err[e]};
          total = tidy(total);
        }
      }
      store(total, b);
    }
    cp_async_wait_all();  // no copy into shared memory outlives the CTA
  } else {
    for (int b = b0; b < blocks; b += stride) {
      Pair sum{0.f, 0.f};
      for (int g = 0; g < groups; ++g) {
        const int64_t j0 = (int64_t)b * size + g * kBlock + lane;  // entries past the end are zeros
        float w[8], err[8];
        weights8<DT, false>(row, (int)(j0 < V ? j0 : V), 32, V, w, err);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = sum + Pair{w[e], err[e]};
        sum = tidy(sum);
      }
      store(sum, b);
    }
  }
  if (!waited) cluster.barrier_wait(std::move(started));
  cluster.sync();
  if (rank != 0) return;
  // the first block whose running sum passes the goal, else the last with weight
  constexpr int kPer = kMaxBlocks / kAccThreads;
  Pair x[kPer], mine{0.f, 0.f};
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    x[e] = tid * kPer + e < blocks ? sums[tid * kPer + e] : Pair{0.f, 0.f};
    mine = mine + x[e];
  }
  const Pair in_warp = scan<32>(mine, lane);
  if (lane == 31) warp_sum[warp] = in_warp;
  __syncthreads();
  // every warp scans the warps' sums
  const Pair all_warps = scan<kAccWarps>(lane < kAccWarps ? warp_sum[lane] : Pair{0.f, 0.f}, lane);
  const Pair whole = shfl(all_warps, kAccWarps - 1);
  const float lift = lift_of(whole);
  const Pair goal = times(u_draw, lift * whole);
  const Pair up_warp = shfl(all_warps, (warp + 31) & 31), up_lane = shfl(in_warp, (lane + 31) & 31);
  Pair run{0.f, 0.f}, last_before{0.f, 0.f};
  if (warp > 0) run = up_warp;
  if (lane > 0) run = run + up_lane;
  int last = -1, first = -1;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const Pair next = run + x[e];
    if (x[e].s > 0.f && first < 0) {
      last = tid * kPer + e;
      last_before = run;
      if (lift * next > goal) first = last;
    }
    run = next;
  }
  // one thread wins: the lowest that found its border, or else the highest with weight
  if (first >= 0) atomicMin(&lowest, tid);
  if (last >= 0) atomicMax(&highest, tid);
  __syncthreads();
  if (tid == (lowest < kAccThreads ? lowest : highest)) {
    pick = last;
    pick_before = last_before;
  }
  __syncthreads();
  int answer;
  if (whole.s > 0.f) {
    const int64_t a = (int64_t)pick * size;
    answer = find_in<DT, VEC>(row, (int)a, (int)(a + size < V ? a + size : V), lift, lift * pick_before, goal, found, warp,
                             lane);
  } else {  // nothing left of the row: all of p
    row.q = nullptr;
    row.n_skip = 0;
    Pair all{0.f, 0.f};
    for (int j0 = warp * kBlock; j0 < V; j0 += kAccWarps * kBlock) {
      float w[8], err[8];
      weights8<DT, VEC>(row, j0 + 8 * lane, 1, V, w, err);
#pragma unroll
      for (int e = 0; e < 8; ++e) all = all + Pair{w[e], 0.f};
      all = tidy(all);
    }
#pragma unroll
    for (int m = 16; m; m >>= 1)
      all = all + Pair{__shfl_xor_sync(0xffffffffu, all.s, m), __shfl_xor_sync(0xffffffffu, all.c, m)};
    if (lane == 0) warp_sum[warp] = all;
    __syncthreads();
    all = warp_sum[0];
#pragma unroll
    for (int g = 1; g < kAccWarps; ++g) all = all + warp_sum[g];
    const float up = lift_of(all);
    answer = find_in<DT, VEC>(row, 0, V, up, Pair{0.f, 0.f}, times(u_draw, up * all), found, warp, lane);
  }
  if (tid == 0) args.next_token[r] = answer;
}

template <int DT, bool TREE>
bool allow_ring() {
  return cudaFuncSetAttribute(accept_kernel<DT, TREE, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kRingBytes<DT>) == cudaSuccess;
}
// The kernels' shared-memory limits, all of them in the first call on a device:
// a later one may be under capture.
kda_status allow_rings() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_CUDA;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
    if (!allow_ring<KDA_DTYPE_F32, false>() || !allow_ring<KDA_DTYPE_F32, true>() ||
        !allow_ring<KDA_DTYPE_BF16, false>() || !allow_ring<KDA_DTYPE_BF16, true>() ||
        !allow_ring<KDA_DTYPE_F16, false>() || !allow_ring<KDA_DTYPE_F16, true>())
      return KDA_ERR_CUDA;
    ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  return KDA_OK;
}

template <int DT, bool TREE, bool VEC>
kda_status launch_accept_kernel(const AcceptArgs& a, cudaLaunchConfig_t cfg) {
  if (VEC) cfg.dynamicSmemBytes = kRingBytes<DT>;
  cudaLaunchKernelEx(&cfg, accept_kernel<DT, TREE, VEC>, a);
  return launch_status();
}

template <int DT>
kda_status launch_accept(const AcceptArgs& a, int B, bool tree, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0 || allow_rings() != KDA_OK) return KDA_ERR_CUDA;
  // CTAs per request: enough to fill the SMs twice, but a block at least for each warp
  int parts = 1;
  while (parts < 8 && (int64_t)B * parts < 2 * sms && (int64_t)parts * kAccWarps * kBlock < a.vocab) parts *= 2;
  // 16-byte loads where every row starts on 16 bytes
  const int64_t es = DT == KDA_DTYPE_F32 ? 4 : 2;
  const bool vec = aligned16(a.target) && a.target_stride * es % 16 == 0 &&
                   (!a.draft || (aligned16(a.draft) && a.draft_stride * es % 16 == 0));
  if ((int64_t)B * parts > INT32_MAX) return KDA_ERR_SHAPE;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(B * parts));
  cfg.blockDim = dim3(kAccThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  record_stage(0, st);
  const kda_status s = tree ? (vec ? launch_accept_kernel<DT, true, true>(a, cfg) : launch_accept_kernel<DT, true, false>(a, cfg))
                            : (vec ? launch_accept_kernel<DT, false, true>(a, cfg) : launch_accept_kernel<DT, false, false>(a, cfg));
  record_stage(1, st);
  record_stage(2, st);
  return s;
}

kda_status accept_common(int dtype, const AcceptArgs& a, int B, bool tree, void* stream) {
  if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F16) return KDA_ERR_UNSUPPORTED;
  if (B < 0 || a.T < 1 || a.vocab < 1 || a.target_stride < a.vocab) return KDA_ERR_SHAPE;
  if (a.T > KDA_ACCEPT_MAX_T || a.vocab > KDA_ACCEPT_MAX_VOCAB) return KDA_ERR_UNSUPPORTED;
  if (a.draft && a.draft_stride < a.vocab) return KDA_ERR_SHAPE;
  if (B == 0) return KDA_OK;
  if (!a.target || !a.tokens || !a.uniforms || !a.accepted || !a.next_token || (tree && (!a.parent || !a.path)))
    return KDA_ERR_NULL_ARG;
  const uintptr_t mask = dtype == KDA_DTYPE_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(a.target) | reinterpret_cast<uintptr_t>(a.draft)) & mask) return KDA_ERR_ALIGNMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == KDA_DTYPE_F32) return launch_accept<KDA_DTYPE_F32>(a, B, tree, st);
  if (dtype == KDA_DTYPE_F16) return launch_accept<KDA_DTYPE_F16>(a, B, tree, st);
  return launch_accept<KDA_DTYPE_BF16>(a, B, tree, st);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_accept_chain(int probs_dtype, const void* target, int64_t target_stride, const void* draft,
                                       int64_t draft_stride, const int32_t* tokens, const float* uniforms,
                                       const int32_t* lengths, int B, int T, int vocab, int32_t* accepted,
                                       int32_t* next_token, int32_t* err_flag, void* stream) {
  AcceptArgs a{};
  a.target = target;
  a.target_stride = target_stride;
  a.draft = draft;
  a.draft_stride = draft_stride;
  a.tokens = tokens;
  a.uniforms = uniforms;
  a.lengths = lengths;
  a.T = T;
  a.vocab = vocab;
  a.accepted = accepted;
  a.next_token = next_token;
  a.err_flag = err_flag;
  return accept_common(probs_dtype, a, B, false, stream);
}

extern "C" kda_status kda_accept_tree(int probs_dtype, const void* target, int64_t target_stride,
                                      const int32_t* tokens, const int32_t* parent_idx, const float* uniforms,
                                      const int32_t* lengths, int B, int T, int vocab, int32_t* accepted,
                                      int32_t* path, int32_t* next_token, int32_t* err_flag, void* stream) {
  AcceptArgs a{};
  a.target = target;
  a.target_stride = target_stride;
  a.tokens = tokens;
  a.parent = parent_idx;
  a.uniforms = uniforms;
  a.lengths = lengths;
  a.T = T;
  a.vocab = vocab;
  a.accepted = accepted;
  a.path = path;
  a.next_token = next_token;
  a.err_flag = err_flag;
  return accept_common(probs_dtype, a, B, true, stream);
}
