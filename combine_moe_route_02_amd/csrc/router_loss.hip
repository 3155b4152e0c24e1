// Auxiliary loss of the router and its gradient: balance loss over packed sequences, z-loss and
// per-expert counts.
//
// Segments s (packed sequences) of counted tokens t; n_s counted tokens, N = sum n_s, S' segments
// with n_s > 0, c_se slots of the top-k at expert e, p_te = softmax(logits_t)_e, lse_t its log-sum:
//   L_bal = 1/S' sum_s E sum_e (c_se / (n_s k)) (sum_t p_te / n_s),  L_z = 1/N sum_t lse_t^2,
//   loss = a L_bal + b L_z.
// Counts carry no gradient, so with w_se = a E c_se / (S' n_s^2 k)
//   dlogits_te = g p_te (w_se - sum_j w_sj p_tj + 2 b lse_t / N).
// The bracket does not change when w_s is shifted, so the kernel takes w_se - a / (S' n_s), formed
// in FP64: near a balanced load every w_se is almost that constant and the difference would lose
// its digits.
//
// Everything is bound by reading the logits once forward and once more (with one write of the
// gradient) backward. A row of E logits is held by 16 to 64 lanes in registers: one pass gives the
// maximum, the sum of exponentials and the probabilities, and each lane adds the probabilities of
// its own columns over the rows it sees, so a tile of rows leaves E partial sums without atomics.
// Tiles never cross a segment; their partials are added in tile order, so results repeat bit for
// bit. Sums over tokens are FP32 inside a tile and FP64 across tiles.
#include "common.h"
#include "launch.h"
#include "trace.h"

namespace moe {

constexpr int kLossThreads = 256;
constexpr int kRedThreads = 1024;
constexpr int kRedCols = 16;                          // columns per reduce block
constexpr int kRedGroups = kRedThreads / kRedCols;    // tiles read side by side

// Rows per tile: about 1024 tiles for long inputs (four 256-thread blocks per CU), down to 32 rows.
int router_loss_tile(int64_t T) {
  int r = 32;
  while (r < 256 && T > (int64_t)r * 1024) r *= 2;
  return r;
}
static int64_t loss_slots(int64_t T, int S) { return T / router_loss_tile(T) + S + 2; }
static int red_blocks(int E) { return (E + kRedCols - 1) / kRedCols; }
static int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

// Workspace: the arrival counter (zero when first used, left zero), then per tile E probability
// sums, E counts, the z sum and the token count, then per segment and reduce block sum_e c P, and
// per segment the z sum.
struct LossWs {
  int* arrived;
  float* p;
  int* c;
  double* z;
  int* n;
  double* cp;
  double* zs;
};
static LossWs loss_ws(void* ws, int64_t T, int S, int E, int64_t* bytes) {
  const int64_t slots = loss_slots(T, S);
  char* b = (char*)ws;
  int64_t at = 0;
  auto take = [&](int64_t n) { char* q = b + at; at += round256(n); return q; };
  LossWs w;
  w.arrived = (int*)take(4);
  w.p = (float*)take(slots * E * 4);
  w.c = (int*)take(slots * E * 4);
  w.z = (double*)take(slots * 8);
  w.n = (int*)take(slots * 4);
  w.cp = (double*)take((int64_t)S * red_blocks(E) * 8);
  w.zs = (double*)take((int64_t)S * 8);
  if (bytes) *bytes = at;
  return w;
}
int64_t router_loss_ws_bytes(int64_t T, int S, int E) {
  int64_t n;
  loss_ws(nullptr, T, S, E, &n);
  return n;
}

// The rows fall into S + 2 pieces: those before the first segment, the segments, those behind the
// last. Piece i starts at bound(i); the tiles of piece i are the blocks from bound(i) / R + i on,
// which leaves room for every piece's rounded-up tile count. Offsets are clamped to [0, T], so a
// bad table gives wrong sums but no access outside the arrays.
struct Pieces {
  const int32_t* off;  // [S + 1] or null: one segment of every row
  int64_t T;
  int S, R;
  MOE_DEV int64_t bound(int i) const {
    if (i == 0 || T == 0) return 0;
    if (i >= S + 2) return T;
    if (!off) return i == 1 ? 0 : T;
    const int64_t o = off[i - 1];
    return o < 0 ? 0 : (o > T ? T : o);
  }
  MOE_DEV int64_t base(int i) const { return bound(i) / R + i; }
};

// The block's piece and rows. Every thread of the block calls it.
struct Tile { int piece; int64_t r0, r1; };
MOE_DEV Tile find_tile(const Pieces& q) {
  const int64_t blk = blockIdx.x;
  int i = -1;
  for (int s0 = 0; s0 < q.S + 2; s0 += kLossThreads) {
    const int s = s0 + (int)threadIdx.x;
    i += __syncthreads_count(s < q.S + 2 && q.base(s) <= blk);
  }
  const int64_t b0 = q.bound(i), b1 = q.bound(i + 1);
  const int64_t r0 = b0 + (blk - q.base(i)) * q.R;
  return {i, r0, b1 < r0 + q.R ? b1 : r0 + q.R};
}

template <int G>
MOE_DEV float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}
template <int G>
MOE_DEV float group_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
  return v;
}

// One row in a group of G lanes: lane q holds columns W * (i * G + q) .. + W of i < NV; columns past
// E hold -inf.
template <int G, int NV, int W>
MOE_DEV void load_row(const float* row, int E, int q, float (&v)[NV * W]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = W * (i * G + q);
    if constexpr (W == 4) {
      const float inf = __builtin_huge_valf();
      const float4 f = e < E ? *(const float4*)(row + e) : make_float4(-inf, -inf, -inf, -inf);
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    } else {
      v[i] = e < E ? row[e] : -__builtin_huge_valf();
    }
  }
}

template <int G, int NV, int W>
__global__ __launch_bounds__(kLossThreads) void router_loss_stats_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
    float* __restrict__ lse_out, Pieces pc, LossWs ws, int E, int K) {
  constexpr int RP = kLossThreads / G;  // rows per pass
  constexpr int C = NV * W;
  __shared__ int hist[1024];
  __shared__ float sums[RP * G * C];
  __shared__ double sz[RP];
  __shared__ int sn[RP];
  const Tile t = find_tile(pc);
  const int tid = threadIdx.x, q = tid % G, g = tid / G;
  if (t.r0 >= t.r1) return;
  if (t.piece == 0 || t.piece == pc.S + 1) {  // rows outside every segment
    for (int64_t r = t.r0 + tid; r < t.r1; r += kLossThreads) lse_out[r] = 0.f;
    return;
  }
  for (int e = tid; e < E; e += kLossThreads) hist[e] = 0;
  __syncthreads();
  float acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
  double z = 0.0;  // lse reaches 1e38 where a row holds the lowest value: its square passes FP32
  int n = 0;
  // every lane runs the same trip count, so the shuffles are never divergent
  for (int64_t rb = t.r0; rb < t.r1; rb += RP) {
    const int64_t r = rb + g;
    const bool in = r < t.r1;
    const bool counted = in && (!mask || mask[r] != 0);
    float v[C];
    int my = -1;
    if (counted) {
      load_row<G, NV, W>(logits + r * E, E, q, v);
      if (q < K) my = idx[r * K + q];
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = -__builtin_huge_valf();
    }
    float m = v[0];
#pragma unroll
    for (int c = 1; c < C; ++c) m = fmaxf(m, v[c]);
    m = group_max<G>(m);
    if (m == -__builtin_huge_valf()) m = 0.f;  // no finite logit: the sum below is 0, or NaN
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      v[c] = __expf(v[c] - m);
      s += v[c];
    }
    s = group_sum<G>(s);
    const bool live = s != 0.f;  // a row of -inf only is left out like a masked one
    const float lse = live ? m + __logf(s) : 0.f;
    const float inv = live ? 1.0f / s : 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = fmaf(v[c], inv, acc[c]);
    z = fma((double)lse, (double)lse, z);
    n += live ? 1 : 0;
    if (in && q == 0) lse_out[r] = lse;
    if (live && my >= 0 && my < E) atomicAdd(&hist[my], 1);
  }
  // sums[g][column as held]: column W * (i * G + q) + w of the lane sits at its own index
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int w = 0; w < W; ++w) sums[g * (G * C) + W * (i * G + q) + w] = acc[i * W + w];
  if (q == 0) { sz[g] = z; sn[g] = n; }
  __syncthreads();
  const int64_t slot = blockIdx.x;
  for (int e = tid; e < E; e += kLossThreads) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < RP; ++k) s += sums[k * (G * C) + e];
    ws.p[slot * E + e] = s;
    ws.c[slot * E + e] = hist[e];
  }
  if (tid == 0) {
    double s = 0.0;
    int m = 0;
#pragma unroll
    for (int k = 0; k < RP; ++k) { s += sz[k]; m += sn[k]; }
    ws.z[slot] = s;
    ws.n[slot] = m;
  }
}

// Adds the tiles of each segment in order: one block per segment and 16 columns, 64 tiles side by
// side. The last block to arrive forms the losses from the segments' sums.
__global__ __launch_bounds__(kRedThreads) void router_loss_reduce_kernel(
    Pieces pc, LossWs ws, int64_t slots, int E, int K, float balance_coef, float z_coef, int32_t* __restrict__ seg_counts,
    int32_t* __restrict__ seg_tokens, float* __restrict__ seg_probs, float* __restrict__ loss) {
  __shared__ double red[kRedThreads];
  __shared__ int redc[kRedThreads];
  __shared__ bool last;
  const int nb = (E + kRedCols - 1) / kRedCols;
  const int s = blockIdx.x / nb, cb = blockIdx.x % nb;
  const int tid = threadIdx.x, col = tid % kRedCols, grp = tid / kRedCols;
  const int e = cb * kRedCols + col;
  const int64_t b0 = pc.bound(s + 1), b1 = pc.bound(s + 2);
  const int64_t first = pc.base(s + 1);
  int64_t end = b1 > b0 ? first + (b1 - b0 + pc.R - 1) / pc.R : first;
  if (end > slots) end = slots;

  double p = 0.0;
  int c = 0;
  if (e < E)
#pragma unroll 4
    for (int64_t i = first + grp; i < end; i += kRedGroups) {
      p += (double)ws.p[i * E + e];
      c += ws.c[i * E + e];
    }
  red[tid] = p;
  redc[tid] = c;
  for (int o = kRedThreads / 2; o >= kRedCols; o >>= 1) {
    __syncthreads();
    if (tid < o) { red[tid] += red[tid + o]; redc[tid] += redc[tid + o]; }
  }
  __syncthreads();
  if (tid < kRedCols && e < E) {
    seg_probs[(int64_t)s * E + e] = (float)red[tid];
    seg_counts[(int64_t)s * E + e] = redc[tid];
  }
  if (tid == 0) {
    double cp = 0.0;
    for (int j = 0; j < kRedCols && cb * kRedCols + j < E; ++j) cp += red[j] * (double)redc[j];
    ws.cp[(int64_t)s * nb + cb] = cp;
  }
  if (cb == 0) {
    __syncthreads();
    double z = 0.0;
    int n = 0;
    for (int64_t i = first + tid; i < end; i += kRedThreads) { z += ws.z[i]; n += ws.n[i]; }
    red[tid] = z;
    redc[tid] = n;
    for (int o = kRedThreads / 2; o > 0; o >>= 1) {
      __syncthreads();
      if (tid < o) { red[tid] += red[tid + o]; redc[tid] += redc[tid + o]; }
    }
    if (tid == 0) { ws.zs[s] = red[0]; seg_tokens[s] = redc[0]; }
  }
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(ws.arrived, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double bal = 0.0, z = 0.0;
  int n = 0, full = 0;
  for (int i = tid; i < pc.S; i += kRedThreads) {
    const int ns = seg_tokens[i];
    if (ns <= 0) continue;
    double cp = 0.0;
    for (int j = 0; j < nb; ++j) cp += ws.cp[(int64_t)i * nb + j];
    bal += cp * (double)E / ((double)ns * (double)ns * (double)K);
    z += ws.zs[i];
    n += ns;
    full += 1;
  }
  __shared__ double redz[kRedThreads];
  __shared__ int redf[kRedThreads];
  red[tid] = bal;
  redz[tid] = z;
  redc[tid] = n;
  redf[tid] = full;
  for (int o = kRedThreads / 2; o > 0; o >>= 1) {
    __syncthreads();
    if (tid < o) {
      red[tid] += red[tid + o];
      redz[tid] += redz[tid + o];
      redc[tid] += redc[tid + o];
      redf[tid] += redf[tid + o];
    }
  }
  if (tid == 0) {
    const double lb = redf[0] ? red[0] / redf[0] : 0.0, lz = redc[0] ? redz[0] / redc[0] : 0.0;
    loss[0] = (float)((double)balance_coef * lb + (z_coef != 0.f ? (double)z_coef * lz : 0.0));  // unused: it may be infinite
    loss[1] = (float)lb;
    loss[2] = (float)lz;
    seg_tokens[pc.S] = redc[0];
    seg_tokens[pc.S + 1] = redf[0];
    *ws.arrived = 0;
  }
}

template <int G, int NV, int W>
__global__ __launch_bounds__(kLossThreads) void router_loss_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ lse_in, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ seg_counts, const int32_t* __restrict__ seg_tokens, const float* __restrict__ dloss,
    float* __restrict__ dlogits, Pieces pc, int E, int K, float balance_coef, float z_coef) {
  constexpr int RP = kLossThreads / G;
  constexpr int C = NV * W;
  const Tile t = find_tile(pc);
  const int tid = threadIdx.x, q = tid % G, g = tid / G;
  if (t.r0 >= t.r1) return;
  const int s = t.piece - 1;
  const bool outside = t.piece == 0 || t.piece == pc.S + 1;
  const int ns = outside ? 0 : seg_tokens[s];
  const int N = seg_tokens[pc.S], full = seg_tokens[pc.S + 1];
  const double per = ns > 0 && full > 0 ? (double)balance_coef / ((double)full * (double)ns) : 0.0;
  const double share = ns > 0 ? (double)E / ((double)ns * (double)K) : 0.0;
  const float zc = N > 0 ? (float)(2.0 * (double)z_coef / (double)N) : 0.f;
  const float gl = dloss ? *dloss : 1.f;
  float w[C];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const int e = W * (i * G + q) + j;
      w[i * W + j] = ns > 0 && e < E ? (float)(per * ((double)seg_counts[(int64_t)s * E + e] * share - 1.0)) : 0.f;
    }
  for (int64_t rb = t.r0; rb < t.r1; rb += RP) {
    const int64_t r = rb + g;
    const bool in = r < t.r1;
    const bool counted = in && !outside && (!mask || mask[r] != 0);
    float v[C], lse = 0.f;
    if (counted) {
      load_row<G, NV, W>(logits + r * E, E, q, v);
      lse = lse_in[r];
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = -__builtin_huge_valf();
    }
    // lse keeps only the digits that its size leaves, up to log E is lost where the logits are huge,
    // so the probabilities are normalised again (the exponent stays within log E of the true one)
    float d = 0.f, sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      v[c] = __expf(v[c] - lse);
      sum += v[c];
      d = fmaf(v[c], w[c], d);
    }
    sum = group_sum<G>(sum);
    d = group_sum<G>(d);
    if (!in) continue;
    const float inv = sum != 0.f ? 1.0f / sum : 0.f;
    const float add = zc * lse - d * inv, scale = gl * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = W * (i * G + q);
      if (e >= E) continue;
      float o[W];
#pragma unroll
      for (int j = 0; j < W; ++j) o[j] = counted ? scale * v[i * W + j] * (w[i * W + j] + add) : 0.f;
      if constexpr (W == 4) *(float4*)(dlogits + r * E + e) = make_float4(o[0], o[1], o[2], o[3]);
      else dlogits[r * E + e] = o[0];
    }
  }
}

// Lanes per row and registers per lane by E: a row of 16-byte vectors in as few lanes as leave one or
// two vectors each (four above 512 experts); rows that are not whole aligned 16-byte vectors go by
// single values.
#define MOE_LOSS_SHAPE(E, vec, ...)                                                             \
  do {                                                                                          \
    if (vec) {                                                                                  \
      if ((E) <= 64) { constexpr int G = 16, NV = 1, W = 4; __VA_ARGS__; }                      \
      else if ((E) <= 128) { constexpr int G = 32, NV = 1, W = 4; __VA_ARGS__; }                \
      else if ((E) <= 256) { constexpr int G = 32, NV = 2, W = 4; __VA_ARGS__; }                \
      else if ((E) <= 512) { constexpr int G = 64, NV = 2, W = 4; __VA_ARGS__; }                \
      else { constexpr int G = 64, NV = 4, W = 4; __VA_ARGS__; }                                \
    } else if ((E) <= 128) { constexpr int G = 64, NV = 2, W = 1; __VA_ARGS__; }                \
    else { constexpr int G = 64, NV = 16, W = 1; __VA_ARGS__; }                                 \
  } while (0)

hipError_t launch_router_loss(const float* logits, const int32_t* topk_idx, const int32_t* seg_offsets,
                              const uint8_t* mask, float* lse, int32_t* seg_counts, int32_t* seg_tokens,
                              float* seg_probs, float* loss, void* workspace, int64_t T, int E, int K, int S,
                              float balance_coef, float z_coef, hipStream_t s) {
  const LossWs ws = loss_ws(workspace, T, S, E, nullptr);
  const Pieces pc{seg_offsets, T, S, router_loss_tile(T)};
  const int64_t slots = loss_slots(T, S);
  if (T > 0) {
    const bool vec = E % 4 == 0 && (uintptr_t)logits % 16 == 0;
    MOE_TRACE("router_loss_stats", s);
    MOE_LOSS_SHAPE(E, vec, MOE_LAUNCH((router_loss_stats_kernel<G, NV, W>), dim3((unsigned)slots), dim3(kLossThreads), 0, s,
                                      logits, topk_idx, mask, lse, pc, ws, E, K));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  {
    MOE_TRACE("router_loss_reduce", s);
    MOE_LAUNCH(router_loss_reduce_kernel, dim3((unsigned)((int64_t)S * red_blocks(E))), dim3(kRedThreads), 0, s, pc, ws,
               slots, E, K, balance_coef, z_coef, seg_counts, seg_tokens, seg_probs, loss);
  }
  return hipGetLastError();
}

hipError_t launch_router_loss_bwd(const float* logits, const float* lse, const int32_t* seg_offsets,
                                  const uint8_t* mask, const int32_t* seg_counts, const int32_t* seg_tokens,
                                  const float* dloss, float* dlogits, int64_t T, int E, int K, int S,
                                  float balance_coef, float z_coef, hipStream_t s) {
  if (T <= 0) return hipSuccess;
  const Pieces pc{seg_offsets, T, S, router_loss_tile(T)};
  const bool vec = E % 4 == 0 && (uintptr_t)logits % 16 == 0 && (uintptr_t)dlogits % 16 == 0;
  {
    MOE_TRACE("router_loss_bwd", s);
    MOE_LOSS_SHAPE(E, vec, MOE_LAUNCH((router_loss_bwd_kernel<G, NV, W>), dim3((unsigned)loss_slots(T, S)),
                                      dim3(kLossThreads), 0, s, logits, lse, mask, seg_counts, seg_tokens, dloss, dlogits,
                                      pc, E, K, balance_coef, z_coef));
  }
  return hipGetLastError();
}

}  // namespace moe
