// Keys that order the experts of a token, and the tile sizes that the routing kernels and the layout kernel share.
#pragma once

#include "common.h"

namespace moe {

constexpr int kRouteBlock = 64;     // tokens per route_layout block (one ballot wave)
constexpr int kRouteThreads = 1024; // route_layout: 16 waves
constexpr int kGroup = 16;          // lanes per token in route_topk
constexpr int kTopkThreads = 256;   // route_topk block
constexpr int kHistTok = kTopkThreads / kGroup;  // tokens per histogram (16)
constexpr int kSub = kRouteBlock / kHistTok;     // histograms per route_layout block (4)

// Order-preserving map of a logit to 32 bits: larger logit -> larger key; NaN ranks as -inf and
// -0 equals +0.
MOE_DEV uint32_t logit_key(float x) {
  if (x != x) x = -__builtin_huge_valf();
  if (x == 0.f) x = 0.f;
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// The same without the two exceptions.
MOE_DEV uint32_t ordered(float x) {
  const int u = __float_as_int(x);
  return (uint32_t)(u ^ ((u >> 31) | (int)0x80000000u));
}
MOE_DEV float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// Full key: logit key above the complemented expert index, so equal logits rank the lower index
// higher. Every real key is > 0; 0 marks an empty list slot.
MOE_DEV uint64_t full_key(float x, int e) {
  return ((uint64_t)logit_key(x) << 32) | (uint32_t)(0xffffffffu - (uint32_t)e);
}

template <int K>
MOE_DEV void insert_key(uint64_t (&l)[K], uint64_t key) {
#pragma unroll
  for (int s = 0; s < K; ++s) {
    const uint64_t cur = l[s];
    const bool take = key > cur;
    l[s] = take ? key : cur;
    key = take ? cur : key;
  }
}

MOE_DEV uint64_t shfl_xor_u64(uint64_t v, int o) {
  const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, o, kWave);
  const uint32_t hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), o, kWave);
  return ((uint64_t)hi << 32) | lo;
}

}  // namespace moe
