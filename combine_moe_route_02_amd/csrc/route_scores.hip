// Routing by scores: softmax or sigmoid of the logits, a balance bias and groups of experts in the choice, gates from
// the chosen scores; the gradient to the logits; the bias update.
//
//   s = sigmoid(l) or softmax(l), c = RN32(s + b) with s in FP64; the topk_groups groups with the largest sums of
//   their group_top largest c are eligible, the k largest c of their experts are chosen (ties: lower index);
//   gate_j = scale s_j, divided by the sum of the chosen s where they are renormalised.
//
// A choice hangs on the last bit of c, so c is defined by FP64 scores, rounded once: two programs, or two kernels,
// that follow the formula choose the same experts.
#include "common.h"
#include "launch.h"
#include "route_keys.h"
#include "trace.h"

namespace moe {

constexpr float kMaxFloat = 3.402823466e38f;
// NaN counts as -inf, +inf as the largest finite value
MOE_DEV float clean_logit(float x) { return x != x ? -__builtin_huge_valf() : fminf(x, kMaxFloat); }

struct ScoreArgs {
  int softmax, groups, keep, top, renorm;
  float scale;
};

MOE_DEV double group16_sum(double x) {
#pragma unroll
  for (int o = kGroup / 2; o > 0; o >>= 1) x += __shfl_xor(x, o, kWave);
  return x;
}

// 16 lanes per token, 16 tokens per workgroup. c of a token's experts goes through LDS for the group sums.
template <int K>
__global__ __launch_bounds__(kTopkThreads) void route_scores_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias, int32_t* __restrict__ topk_idx,
    float* __restrict__ gates, int32_t* __restrict__ block_hist, int64_t T, int E, int n, int chunk0, int nbpc,
    ScoreArgs a) {
  extern __shared__ int smem[];  // [E] histogram, [16][E] c
  int* hist = smem;
  const int tid = threadIdx.x, q = tid & (kGroup - 1), tl = tid / kGroup;
  float* c = (float*)(smem + E) + tl * E;
  const int ch = chunk0 + blockIdx.x / nbpc;
  const int bl = blockIdx.x % nbpc;
  const ChunkRange cr = chunk_range(T, n, ch);
  for (int e = tid; e < E; e += kTopkThreads) hist[e] = 0;
  __syncthreads();
  const int64_t t = cr.t0 + (int64_t)bl * kHistTok + tl;
  const bool valid = t < cr.t1;
  const float* row = logits + (valid ? t : 0) * (int64_t)E;
  float m = -__builtin_huge_valf();
  double den = 1.0;
  if (a.softmax) {
    if (valid) for (int e = q; e < E; e += kGroup) m = fmaxf(m, clean_logit(row[e]));
#pragma unroll
    for (int o = kGroup / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
    den = 0.0;
    if (valid && m > -__builtin_huge_valf())
      for (int e = q; e < E; e += kGroup) den += exp((double)clean_logit(row[e]) - (double)m);
    den = group16_sum(den);
  }
  if (valid)
    for (int e = q; e < E; e += kGroup) {
      const double l = clean_logit(row[e]);
      const double s = !a.softmax ? 1.0 / (1.0 + exp(-l)) : den > 0.0 ? exp(l - (double)m) / den : 0.0;
      const float x = (float)(bias ? s + (double)bias[e] : s);
      c[e] = x != x ? -__builtin_huge_valf() : x;
    }
  __syncthreads();
  uint64_t kept = ~0ull;
  const int gs = E / a.groups;
  if (a.groups > 1) {
    uint32_t mine[4];  // keys of groups q, q + 16, ...
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int g = q + kGroup * u;
      mine[u] = 0;
      if (valid && g < a.groups) {
        float b0 = -__builtin_huge_valf(), b1 = b0;
        for (int e = g * gs; e < (g + 1) * gs; ++e) {
          const float x = c[e];
          b1 = fmaxf(b1, fminf(b0, x));
          b0 = fmaxf(b0, x);
        }
        mine[u] = logit_key(a.top == 2 && gs > 1 ? b0 + b1 : b0);
      }
    }
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int g = q + kGroup * u;
      if (kGroup * u >= a.groups) break;
      int beaten = 0;
      for (int o = 0; o < a.groups; ++o) {
        // group o's key is in lane o % 16 of the token's lanes, entry o / 16
        const uint32_t k0 = (uint32_t)__shfl((int)mine[0], o & 15, kGroup), k1 = (uint32_t)__shfl((int)mine[1], o & 15, kGroup);
        const uint32_t k2 = (uint32_t)__shfl((int)mine[2], o & 15, kGroup), k3 = (uint32_t)__shfl((int)mine[3], o & 15, kGroup);
        const uint32_t other = o < 16 ? k0 : o < 32 ? k1 : o < 48 ? k2 : k3;
        beaten += other > mine[u] || (other == mine[u] && o < g);
      }
      if (g < a.groups && beaten < a.keep) { if (g < 32) lo |= 1u << g; else hi |= 1u << (g - 32); }
    }
#pragma unroll
    for (int o = kGroup / 2; o > 0; o >>= 1) {
      lo |= (uint32_t)__shfl_xor((int)lo, o, kWave);
      hi |= (uint32_t)__shfl_xor((int)hi, o, kWave);
    }
    kept = ((uint64_t)hi << 32) | lo;
  }
  uint64_t l[K], sel[K];
#pragma unroll
  for (int s = 0; s < K; ++s) l[s] = 0;
  if (valid)
    for (int e = q; e < E; e += kGroup)
      if ((kept >> (e / gs)) & 1) insert_key<K>(l, full_key(c[e], e));
#pragma unroll
  for (int s = 0; s < K; ++s) {
    uint64_t best = l[0];
#pragma unroll
    for (int o = kGroup / 2; o > 0; o >>= 1) {
      const uint64_t other = shfl_xor_u64(best, o);
      best = other > best ? other : best;
    }
    sel[s] = best;
    if (l[0] == best) {
#pragma unroll
      for (int r = 0; r + 1 < K; ++r) l[r] = l[r + 1];
      l[K - 1] = 0;
    }
  }
  if (valid && q < K) {
    // gates, computed relative to the largest so that the sum of very small scores keeps its digits
    float top = -__builtin_huge_valf(), mine = 0.f, sum = 0.f;
    int id = 0;
    float z[K];
#pragma unroll
    for (int s = 0; s < K; ++s) {
      const int e = (int)(0xffffffffu - (uint32_t)sel[s]);
      if (s == q) id = e;
      z[s] = clean_logit(row[e]);
      top = fmaxf(top, a.softmax ? z[s] : fminf(z[s], 0.f));
    }
    float g;
    if (a.renorm) {
#pragma unroll
      for (int s = 0; s < K; ++s) {
        float u = 0.f;
        if (top > -__builtin_huge_valf())
          u = a.softmax ? expf(z[s] - top) : expf(fminf(z[s], 0.f) - top) / (1.f + expf(-fabsf(z[s])));
        sum += u;
        if (s == q) mine = u;
      }
      g = sum > 0.f ? mine / sum : 0.f;
    } else {
      float zq = 0.f;
#pragma unroll
      for (int s = 0; s < K; ++s) if (s == q) zq = z[s];
      if (a.softmax) g = den > 0.0 ? expf(zq - m) / (float)den : 0.f;
      else g = expf(fminf(zq, 0.f)) / (1.f + expf(-fabsf(zq)));
    }
    topk_idx[t * K + q] = id;
    gates[t * K + q] = a.scale * g;
    atomicAdd(&hist[id], 1);
  }
  __syncthreads();
  int32_t* out = block_hist + (int64_t)ch * E * nbpc + bl;
  for (int e = tid; e < E; e += kTopkThreads) out[(int64_t)e * nbpc] = hist[e];
}

// Gradient to the logits, one wave per token. With gh_j = s_j / sum s over the chosen experts:
//   sigmoid: dl_j = scale gh_j (1 - s_j)(dg_j - sum gh_i dg_i), or scale s_j (1 - s_j) dg_j where gates are not renormalised
//   softmax: dl_j = scale gh_j (dg_j - sum gh_i dg_i), or, for every expert, scale p_e ([e = idx_j] dg_j - sum p_i dg_i)
// 1 - s_j is taken as sigmoid(-l_j). ADD: dlogits holds another term. The planes are route_bwd_dlogits'.
template <bool ADD>
__global__ __launch_bounds__(256) void route_scores_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ dgates, const int32_t* __restrict__ idx,
    float* __restrict__ dlogits, uint16_t* __restrict__ dl_hi, uint16_t* __restrict__ dl_lo, int ldl, int64_t pitch,
    int64_t t0, int64_t t1, int K, int E, ScoreArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = t0 + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= t1) return;
  const float ninf = -__builtin_huge_valf();
  const float* lr = logits + t * (int64_t)E;
  float* row = dlogits + t * (int64_t)E;
  const bool dense = a.softmax && !a.renorm;
  const int id = lane < K ? idx[t * K + lane] : -1;
  const float d = lane < K ? dgates[t * K + lane] : 0.f;
  const float z = lane < K ? clean_logit(lr[id]) : ninf;
  float v = 0.f, m = ninf, inv = 0.f, mean = 0.f;
  if (dense) {
    for (int e = lane; e < E; e += 64) m = fmaxf(m, clean_logit(lr[e]));
    m = wave_max(m);
    float s = 0.f;
    if (m > ninf) for (int e = lane; e < E; e += 64) s += expf(clean_logit(lr[e]) - m);
    s = wave_sum(s);
    inv = s > 0.f ? 1.f / s : 0.f;
    const float p = lane < K && m > ninf ? expf(z - m) * inv : 0.f;
    mean = wave_sum(p * d);
    v = a.scale * p * d;  // added to -scale p mean below
  } else if (a.renorm) {
    const float top = wave_max(a.softmax ? z : fminf(z, 0.f));
    float u = 0.f;
    if (lane < K && top > ninf)
      u = a.softmax ? expf(z - top) : expf(fminf(z, 0.f) - top) / (1.f + expf(-fabsf(z)));
    const float s = wave_sum(u);
    const float gh = s > 0.f ? u / s : 0.f;
    const float rest = a.softmax ? 1.f : expf(-fmaxf(z, 0.f)) / (1.f + expf(-fabsf(z)));
    v = a.scale * gh * rest * (d - wave_sum(gh * d));
  } else {
    const float e1 = expf(-fabsf(z));
    v = a.scale * d * e1 / ((1.f + e1) * (1.f + e1));  // s (1 - s)
  }
  float vs[8];
  int ids[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    ids[j] = j < K ? __shfl(id, j, 64) : -1;
    vs[j] = j < K ? __shfl(v, j, 64) : 0.f;
  }
  auto value = [&](int e) {
    float x = dense && m > ninf ? -a.scale * mean * (expf(clean_logit(lr[e]) - m) * inv) : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) if (ids[j] == e) x += vs[j];
    if constexpr (ADD) x += row[e];
    return x;
  };
  if (!dl_hi) {
    for (int e = lane; e < E; e += 64) row[e] = value(e);
    return;
  }
  // two columns per lane (E is a multiple of 4 where planes are written), zeros past E
  uint32_t* hr = (uint32_t*)(dl_hi + (t - t0) * pitch);
  uint32_t* lp = (uint32_t*)(dl_lo + (t - t0) * pitch);
  for (int e = 2 * lane; e < ldl; e += 128) {
    float x0 = 0.f, x1 = 0.f;
    if (e < E) {
      x0 = value(e);
      x1 = value(e + 1);
      *(float2*)(row + e) = make_float2(x0, x1);
    }
    const uint16_t h0 = f2bf(x0), h1 = f2bf(x1);
    hr[e / 2] = (uint32_t)h0 | ((uint32_t)h1 << 16);
    lp[e / 2] = (uint32_t)f2bf(x0 - bf2f(h0)) | ((uint32_t)f2bf(x1 - bf2f(h1)) << 16);
  }
}

// b_e += rate sign(mean count - count_e), from the sign of sum count - E count_e in 64-bit integers.
__global__ __launch_bounds__(256) void router_bias_update_kernel(int E, int rows, const int32_t* __restrict__ counts,
                                                                 float rate, float* __restrict__ bias) {
  __shared__ long long part[4];
  long long sum = 0;
  for (int64_t i = threadIdx.x; i < (int64_t)rows * E; i += 256) sum += counts[i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = part[0] + part[1] + part[2] + part[3];
  for (int e = threadIdx.x; e < E; e += 256) {
    long long own = 0;
    for (int r = 0; r < rows; ++r) own += counts[(int64_t)r * E + e];
    const long long d = sum - (long long)E * own;
    bias[e] += d > 0 ? rate : d < 0 ? -rate : 0.f;
  }
}

static ScoreArgs score_args(const moe_router_scores& r) {
  return {r.score == MOE_SCORE_SOFTMAX, r.n_groups, r.topk_groups, r.group_top, r.renormalize != 0, r.scale};
}

hipError_t launch_route_scores(const moe_router_scores& r, const float* logits, const float* bias, int32_t* topk_idx,
                               float* gates, int32_t* counts, int32_t* offsets, int32_t* row_of, int32_t* src_token,
                               int32_t* scratch, int64_t T, int E, int e0, int El, int K, int n, int chunk0, int nchunks,
                               int64_t P_c, hipStream_t s) {
  const int nbpc = route_blocks_per_chunk(T, n) * kSub;
  const size_t lds = (size_t)E * (1 + kHistTok) * 4;
  {
    MOE_TRACE("route_scores", s);
    switch (K) {
#define MOE_RS_K(KK)                                                                                              \
  case KK: {                                                                                                      \
    auto k = route_scores_kernel<KK>;                                                                             \
    if (lds > 65536) {                                                                                            \
      hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);   \
      if (e != hipSuccess) return e;                                                                              \
    }                                                                                                             \
    MOE_LAUNCH(k, dim3(nbpc * nchunks), dim3(kTopkThreads), lds, s, logits, bias, topk_idx, gates, scratch, T, E, \
               n, chunk0, nbpc, score_args(r));                                                                   \
    break;                                                                                                        \
  }
      MOE_RS_K(1) MOE_RS_K(2) MOE_RS_K(3) MOE_RS_K(4) MOE_RS_K(5) MOE_RS_K(6) MOE_RS_K(7) MOE_RS_K(8)
#undef MOE_RS_K
      default: return hipErrorInvalidValue;
    }
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  return launch_layout(topk_idx, scratch, counts, offsets, row_of, src_token, T, E, e0, El, K, n, chunk0, nchunks, P_c, s);
}

hipError_t launch_route_scores_bwd(const moe_router_scores& r, const float* logits, const float* dgates,
                                   const int32_t* idx, float* dlogits, int64_t t0, int64_t t1, int K, int E,
                                   hipStream_t s, uint16_t* dl_hi, uint16_t* dl_lo, int ldl, int64_t pitch, bool add) {
  if (dl_hi && (!dl_lo || E % 2 || ldl < E || ldl % 8 || pitch % 2 || pitch < ldl)) return hipErrorInvalidValue;
  if (t1 <= t0) return hipSuccess;
  MOE_TRACE("route_scores_bwd", s);
  auto k = add ? route_scores_bwd_kernel<true> : route_scores_bwd_kernel<false>;
  MOE_LAUNCH(k, dim3((unsigned)((t1 - t0 + 3) / 4)), dim3(256), 0, s, logits, dgates, idx, dlogits, dl_hi, dl_lo, ldl,
             pitch, t0, t1, K, E, score_args(r));
  return hipGetLastError();
}

hipError_t launch_router_bias_update(int E, int rows, const int32_t* counts, float rate, float* bias, hipStream_t s) {
  MOE_TRACE("router_bias_update", s);
  MOE_LAUNCH(router_bias_update_kernel, dim3(1), dim3(256), 0, s, E, rows, counts, rate, bias);
  return hipGetLastError();
}

}  // namespace moe
