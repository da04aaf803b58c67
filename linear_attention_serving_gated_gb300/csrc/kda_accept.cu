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
// Accept tests are exact: the product of two FP32 numbers fits FP64.  A
// thread's sum of weights is an FP32 pair (sum, error) whose error part takes
// what each addition and each difference p - q rounds off (two-sum; 48 bits),
// and pairs are joined in FP64; FP64 for every element would be bound by its
// rate, 1/64 of FP32's here.  The whole is the last of the running sums.
//
// One cluster per request: every CTA repeats the walk (a few gathered loads,
// whose latency is the same for one CTA as for all), sums a contiguous part
// of the row and stores one FP64 sum per warp in the first CTA's shared
// memory.  The first CTA's first warp finds the warp part that holds the
// border and goes through that part again, 32 lanes at a time.
#include <cooperative_groups.h>

#include "kda_host.h"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kAccThreads = 256, kAccWarps = kAccThreads / 32;
constexpr int kMaxCluster = 16;

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
  const void* q;        // nullptr: no draft row
  int64_t p0, q0;       // element offsets of the rows
  const int* skip;      // tokens that fell
  int n_skip;
};

template <int DT>
__device__ __forceinline__ double weight_at(const Row& r, int j) {
  const float p = prob_at<DT>(r.p, r.p0 + j);
  if (r.q) {
    const float q = prob_at<DT>(r.q, r.q0 + j);
    return p > q ? (double)p - (double)q : 0.0;
  }
  for (int s = 0; s < r.n_skip; ++s)
    if (r.skip[s] == j) return 0.0;
  return p;
}

__device__ __forceinline__ double warp_scan(double x, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// The lowest j in [lo, hi) with weight whose running sum from `before` exceeds
// `goal`; where rounding leaves none, the last j with weight; -1 where none has
// any.  One warp: first 32 equal pieces, then the elements of one.
template <int DT>
__device__ int find_in(const Row& row, int lo, int hi, double before, double goal, int lane) {
  const int piece = (hi - lo + 31) / 32;
  int a = min(lo + lane * piece, hi), b = min(a + piece, hi);
  double s = 0.0;
  for (int j = a; j < b; ++j) s += weight_at<DT>(row, j);
  const double cum = before + warp_scan(s, lane);
  const unsigned some = __ballot_sync(0xffffffffu, s > 0.0);
  const unsigned over = __ballot_sync(0xffffffffu, s > 0.0 && cum > goal);
  if (!some) return -1;
  const int L = over ? __ffs(over) - 1 : 31 - __clz(some);
  double base = __shfl_sync(0xffffffffu, cum - s, L);
  a = __shfl_sync(0xffffffffu, a, L);
  b = __shfl_sync(0xffffffffu, b, L);
  int last = -1;
  for (int j0 = a; j0 < b; j0 += 32) {
    const double w = j0 + lane < b ? weight_at<DT>(row, j0 + lane) : 0.0;
    const double c = base + warp_scan(w, lane);
    const unsigned pos = __ballot_sync(0xffffffffu, w > 0.0);
    const unsigned o = __ballot_sync(0xffffffffu, w > 0.0 && c > goal);
    if (o) return j0 + __ffs(o) - 1;
    if (pos) last = j0 + 31 - __clz(pos);
    base = __shfl_sync(0xffffffffu, c, 31);
  }
  return last;
}

template <int DT, bool TREE>
__global__ void __launch_bounds__(kAccThreads) accept_kernel(const AcceptArgs args) {
  cg::cluster_group cluster = cg::this_cluster();
  auto started = cluster.barrier_arrive();
  const int rank = cluster.block_rank(), parts = cluster.num_blocks();
  const int r = blockIdx.x / parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = args.T, V = args.vocab;
  __shared__ float p_tok[KDA_ACCEPT_MAX_T];
  __shared__ int tok_s[KDA_ACCEPT_MAX_T], par_s[TREE ? KDA_ACCEPT_MAX_T : 1], skip_s[KDA_ACCEPT_MAX_T];
  __shared__ float u_s[TREE ? KDA_ACCEPT_MAX_T : 1];
  __shared__ double sums[kMaxCluster * kAccWarps];
  __shared__ int first_fall, cur_s, n_skip_s;

  const int64_t r0 = (int64_t)r * T;
  int n = args.lengths ? args.lengths[r] : T;
  const bool report = rank == 0 && tid == 0;
  if (n < 0 || n > T) {
    if (report) set_error(args.err_flag, KDA_DEVERR_SEQLENS);
    n = 0;
  }
  if (tid == 0) {
    first_fall = n;
    n_skip_s = 0;
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
  for (int i = 1 + tid; i < n; i += kAccThreads) {
    const int tok = args.tokens[r0 + i];
    const bool in = tok >= 0 && tok < V;
    if (!in && rank == 0) set_error(args.err_flag, KDA_DEVERR_TOKEN);
    const int up = TREE ? par_s[i] : i - 1;
    const float p = in ? prob_at<DT>(args.target, (r0 + up) * args.target_stride + tok) : 0.f;
    const float u = args.uniforms[r0 + i];
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
  if (tid == 0) {
    int cur = first_fall - 1;
    if constexpr (TREE) {
      // children follow their parents, so one pass over the nodes is the walk
      cur = 0;
      int n_skip = 0, depth = 0;
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
    } else if (!args.draft && cur + 1 < n) {
      skip_s[0] = args.tokens[r0 + cur + 1];
      n_skip_s = 1;
    }
    cur_s = cur;
    if (report) args.accepted[r] = n > 0 ? cur : -1;
  }
  __syncthreads();
  const int cur = cur_s;
  if (n == 0) {  // the same for every CTA of the cluster
    cluster.barrier_wait(std::move(started));
    if (report) args.next_token[r] = -1;
    return;
  }
  Row row{args.target, nullptr, (r0 + cur) * args.target_stride, 0, skip_s, n_skip_s};
  if (!TREE && args.draft && cur + 1 < n) {
    row.q = args.draft;
    row.q0 = ((int64_t)r * (T - 1) + cur) * args.draft_stride;
  }
  // this warp's part of the row
  const int per_warp = (V + parts * kAccWarps - 1) / (parts * kAccWarps);
  const int64_t at = (int64_t)(rank * kAccWarps + warp) * per_warp;
  const int lo = (int)(at < V ? at : V), hi = (int)(at + per_warp < V ? at + per_warp : V);
  float s = 0.f, c = 0.f;
  for (int j = lo + lane; j < hi; j += 32) {
    const float p = prob_at<DT>(row.p, row.p0 + j);
    float w = p, e = 0.f;
    if (row.q) {
      const float q = prob_at<DT>(row.q, row.q0 + j);
      w = p - q;
      const float b = p - w;  // q as subtracted; p - q = w + e exactly
      e = (p - (w + b)) + (b - q);
      if (!(p > q)) w = e = 0.f;
    } else {
      for (int k = 0; k < row.n_skip; ++k)
        if (row.skip[k] == j) w = 0.f;
    }
    const float t = s + w, z = t - s;
    c += (s - (t - z)) + (w - z) + e;
    s = t;
  }
  double sum = (double)s + (double)c;
#pragma unroll
  for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  // every CTA of the cluster has started: its shared memory may be written
  cluster.barrier_wait(std::move(started));
  if (lane == 0) *cluster.map_shared_rank(&sums[rank * kAccWarps + warp], 0) = sum;
  cluster.sync();
  if (rank != 0 || warp != 0) return;
  const int blocks = parts * kAccWarps;
  double whole = 0.0;
  for (int b0 = 0; b0 < blocks; b0 += 32)
    whole = __shfl_sync(0xffffffffu, whole + warp_scan(b0 + lane < blocks ? sums[b0 + lane] : 0.0, lane), 31);
  const double u = args.uniforms[r0];
  int answer = -1;
  if (whole > 0.0) {
    const double goal = u * whole;
    int part = 0;  // the first part whose running sum passes the goal, else the last with weight
    double before = 0.0, part_before = 0.0;
    for (int b0 = 0; b0 < blocks; b0 += 32) {
      const double x = b0 + lane < blocks ? sums[b0 + lane] : 0.0;
      const double cum = before + warp_scan(x, lane);
      const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
      const unsigned over = __ballot_sync(0xffffffffu, x > 0.0 && cum > goal);
      if (some) {
        const int pick = over ? __ffs(over) - 1 : 31 - __clz(some);
        part = b0 + pick;
        part_before = __shfl_sync(0xffffffffu, cum - x, pick);
      }
      if (over) break;
      before = __shfl_sync(0xffffffffu, cum, 31);
    }
    const int64_t p0 = (int64_t)part * per_warp;
    answer = find_in<DT>(row, (int)p0, (int)(p0 + per_warp < V ? p0 + per_warp : V), part_before, goal, lane);
  } else {  // nothing left of the row: all of p
    row.q = nullptr;
    row.n_skip = 0;
    double all = 0.0;
    for (int j = lane; j < V; j += 32) all += weight_at<DT>(row, j);
#pragma unroll
    for (int m = 16; m; m >>= 1) all += __shfl_xor_sync(0xffffffffu, all, m);
    answer = find_in<DT>(row, 0, V, 0.0, u * all, lane);
  }
  if (lane == 0) args.next_token[r] = answer;
}

template <int DT>
kda_status launch_accept(const AcceptArgs& a, int B, bool tree, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0) return KDA_ERR_CUDA;
  // CTAs per request: enough to fill the SMs twice, but at least 128 elements a warp
  int parts = 1;
  while (parts < 8 && (int64_t)B * parts < 2 * sms && (int64_t)parts * kAccWarps * 128 < a.vocab) parts *= 2;
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
  cudaLaunchKernelEx(&cfg, tree ? accept_kernel<DT, true> : accept_kernel<DT, false>, a);
  const kda_status s = launch_status();
  record_stage(1, st);
  record_stage(2, st);
  return s;
}

kda_status accept_common(int dtype, const AcceptArgs& a, int B, bool tree, void* stream) {
  if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F16) return KDA_ERR_UNSUPPORTED;
  if (B < 0 || a.T < 1 || a.vocab < 1 || a.target_stride < a.vocab) return KDA_ERR_SHAPE;
  if (a.T > KDA_ACCEPT_MAX_T) return KDA_ERR_UNSUPPORTED;
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
