// route_token.hpp -- one token's top-k selection and renormalised softmax
// weights by a group of lanes, shared by the routing kernels and the layer for
// a few tokens (route.hip states the selection rule and the design).
#pragma once

#include "common.hpp"

namespace tre {

// Unsigned order of a float32: larger float -> larger integer; -0.0 is
// mapped to +0.0 first so that the two compare equal.
__device__ __forceinline__ uint32_t float_order(float f) {
  uint32_t u = __builtin_bit_cast(uint32_t, f);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float order_to_float(uint32_t o) {
  uint32_t u = (o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o;
  return __builtin_bit_cast(float, u);
}

// Key of expert e: nonzero for every real expert, so 0 marks "none".
__device__ __forceinline__ uint64_t make_key(float logit, int e) {
  return ((uint64_t)float_order(logit) << 32) | (uint64_t)(0xFFFFFFFFu - (uint32_t)e);
}

template <int G>
__device__ __forceinline__ uint64_t group_max(uint64_t v) {
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) {
    uint32_t lo = __shfl_xor((uint32_t)v, off, G);
    uint32_t hi = __shfl_xor((uint32_t)(v >> 32), off, G);
    uint64_t o = ((uint64_t)hi << 32) | lo;
    v = o > v ? o : v;
  }
  return v;
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, G);
  return v;
}

// Route token t from this lane's logits lg[s] = logit of expert s * G + lane
// (a group of G lanes per token; the group is wholly active or wholly idle).
template <int G, int S>
__device__ __forceinline__ void route_token(const float (&lg)[S], int64_t t, bool active, int E, int k,
                                            int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  const int lane = threadIdx.x % G;
  uint64_t key[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = s * G + lane;
    key[s] = (active && e < E) ? make_key(lg[s], e) : 0ull;
  }

  uint64_t sel[S];  // pick j is held by lane j % G in slot j / G
#pragma unroll
  for (int s = 0; s < S; ++s) sel[s] = 0ull;
  uint64_t first = 0ull;
  for (int j = 0; j < k; ++j) {
    uint64_t best = 0ull;
#pragma unroll
    for (int s = 0; s < S; ++s) best = key[s] > best ? key[s] : best;
    best = group_max<G>(best);
    if (j == 0) first = best;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (key[s] == best) key[s] = 0ull;
      if (s == j / G && lane == j % G) sel[s] = best;
    }
  }
  if (!active) return;

  const float m = order_to_float((uint32_t)(first >> 32));
  float p[S];
  float local = 0.f;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const bool mine = s * G + lane < k;
    p[s] = mine ? expf(order_to_float((uint32_t)(sel[s] >> 32)) - m) : 0.f;
    local += p[s];
  }
  const float z = group_sum<G>(local);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int j = s * G + lane;
    if (j < k) {
      topk_idx[t * k + j] = (int32_t)(0xFFFFFFFFu - (uint32_t)sel[s]);
      topk_w[t * k + j] = p[s] / z;
    }
  }
}

}  // namespace tre
