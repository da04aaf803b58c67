// lin.cuh -- the decay of linear attention with one decay per value head.
#pragma once

#include "kda_host.h"

namespace kda {

struct LinGateArgs {
  const float* A_log;    // [HV] or nullptr: the gate input is the FP32 log-decay
  const float* dt_bias;  // [HV] or nullptr
  const void* a;         // gate input [rows, HV], or nullptr: every token decays by -exp(A_log)
  int use_qk_l2norm;
  float scale;
};

inline kda_status check_lin_gate(const kda_scalar_gate& g, const void* a, LinGateArgs* out) {
  if (!a && !g.A_log) return KDA_ERR_NULL_ARG;
  // the gate input is read one element at a time, so it needs only its own alignment
  if (reinterpret_cast<uintptr_t>(a) & (g.A_log ? 1u : 3u)) return KDA_ERR_ALIGNMENT;
  out->A_log = g.A_log;
  out->dt_bias = g.A_log && a ? g.dt_bias : nullptr;
  out->a = a;
  out->use_qk_l2norm = g.use_qk_l2norm;
  out->scale = g.scale;
  return KDA_OK;
}

// The gate input of one token and head, loaded without a branch on its type, so
// that other loads need not wait for its outcome.
__device__ __forceinline__ ushort2 lin_gate_load(const LinGateArgs& ga, int64_t at) {
  if (!ga.a) return make_ushort2(0, 0);
  const bool raw = ga.A_log != nullptr;
  const uint16_t* p = static_cast<const uint16_t*>(ga.a) + (raw ? at : 2 * at);
  return make_ushort2(__ldg(p), __ldg(p + (raw ? 0 : 1)));
}

// Its log-decay: -exp(A_log) softplus(a + dt_bias), given, or -exp(A_log);
// neg_rate = -exp(A_log[h]), bias = dt_bias[h].  Below -128 the factor is zero in
// FP32 and stays zero in any sum with others, and above 0 a state would grow: the
// cuts keep sums finite and let a NaN through.
template <bool F16>
__device__ __forceinline__ float lin_log_decay(const LinGateArgs& ga, ushort2 in, float neg_rate, float bias) {
  float g = neg_rate;
  if (ga.a) {
    if (ga.A_log) {
      const float x = in16_to_float<F16>(in.x) + bias;
      g = neg_rate * (x > 20.f ? x : log1pf(expf(x)));  // softplus; past 20 it is x to 2^-28
    } else {
      g = __uint_as_float((uint32_t)in.y << 16 | in.x);
    }
  }
  return g < -128.f ? -128.f : g > 0.f ? 0.f : g;
}

}  // namespace kda
