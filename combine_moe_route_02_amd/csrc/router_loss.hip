// Auxiliary loss of the router and its gradient: balance loss over packed sequences, z-loss and
// per-expert counts.
//
// Segments s (packed sequences) of counted tokens t; n_s counted tokens, N = sum n_s, S' segments
// with n_s > 0, c_se slots of the top-k at expert e, p_te = softmax(logits_t)_e, lse_t its log-sum:
//   L_bal = 1/S' sum_s E sum_e (c_se / (n_s k)) (sum_t p_te / n_s),  L_z = 1/N sum_t lse_t^2,
//   loss = a L_bal + b L_z.
// Counts carry no gradient, so with w_se = a E c_se / (S' n_s^2 k)
//   dlogits_te = g p_te (w_se - sum_j w_sj p_tj + 2 b lse_t / N).
// The bracket does not change when w_s is shifted, so the kernel takes w_se - a / (S' n_s) =
// a (c_se E - n_s k) / (S' n_s^2 k), the difference in integers: near a balanced load every w_se is almost
// that constant and a difference of the two in floating point would lose its digits.
//
// Everything is bound by reading the logits once forward and once more (with one write of the
// gradient) backward. A row of E logits is held by 8 to 64 lanes in registers: one pass gives the
// maximum, the sum of exponentials and the probabilities, and each lane adds the probabilities of
// its own columns over the rows it sees, so a tile of rows leaves E partial sums without atomics.
// 131072 tokens of 256 experts: forward 27 us (5.0 TB/s), sums 10 us, backward 45 us (268 MB); 512 tokens 4.8 + 4.4 +
// 5.2 us, latency of three launches.
// Tiles never cross a segment; their partials are added in tile order, so results repeat bit for
// bit. Sums over tokens are FP32 inside a tile and FP64 across tiles.
#include "common.h"
#include "launch.h"
#include "trace.h"

namespace moe {

constexpr int kLossThreads = 256;
constexpr int kRedThreads = 1024;
constexpr int kRedCols = 16;  // columns per reduce block (the fewest)

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
  int S, R;  // R rows per tile, 2^shift
  int shift;
  MOE_DEV int64_t bound(int i) const {
    if (i == 0 || T == 0) return 0;
    if (i >= S + 2) return T;
    if (!off) return i == 1 ? 0 : T;
    const int64_t o = off[i - 1];
    return o < 0 ? 0 : (o > T ? T : o);
  }
  MOE_DEV int64_t base(int i) const { return (bound(i) >> shift) + i; }
};

// The block's piece and rows. Every thread of the block calls it. Every block scans the segments, so the time grows with
// their square once they are many: 131072 tokens of 128 experts, forward and backward, 53 us with up to 64 segments, 118 us
// with 1024, 0.7 ms with 8192, 15 ms with 65536.
struct Tile { int piece; int64_t r0, r1; };
MOE_DEV Tile find_tile(const Pieces& q) {
  const int64_t blk = blockIdx.x;
  if (!q.off) {  // one segment: pieces 0 and 2 are empty, block 0 has no tile
    const int64_t r0 = (blk - 1) * q.R;
    return {1, blk > 0 ? r0 : q.T, q.T < r0 + q.R ? q.T : r0 + q.R};
  }
  int i = -1;
  for (int s0 = 0; s0 < q.S + 2; s0 += kLossThreads) {
    const int s = s0 + (int)threadIdx.x;
    i += __syncthreads_count(s < q.S + 2 && q.base(s) <= blk);
  }
  const int64_t b0 = q.bound(i), b1 = q.bound(i + 1);
  const int64_t r0 = b0 + (blk - q.base(i)) * q.R;
  return {i, r0, b1 < r0 + q.R ? b1 : r0 + q.R};
}

// Reductions over aligned groups of G lanes, every lane getting the result: DPP steps inside 16 lanes
// (quad permutes, then mirrors of 8 and of 16), gfx950's row and half swaps above. A shuffle through
// LDS takes several times a DPP step, and a row has two such chains.
template <int CTRL>
MOE_DEV float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int G, class Op>
MOE_DEV float group_reduce(float v, Op&& op) {
  v = op(v, dpp<0xB1>(v));   // lane ^ 1
  v = op(v, dpp<0x4E>(v));   // lane ^ 2
  v = op(v, dpp<0x141>(v));  // mirror of 8 lanes
  if constexpr (G >= 16) v = op(v, dpp<0x140>(v));  // mirror of 16 lanes
  if constexpr (G >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (G >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
template <int G>
MOE_DEV float group_sum(float v) { return group_reduce<G>(v, [](float a, float b) { return a + b; }); }
template <int G>
MOE_DEV float group_max(float v) { return group_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); }); }

// One row in a group of G lanes: lane q holds columns W * (i * G + q) .. + W of i < NV. Loads carry no branch
// (behind one the compiler waits for every load in flight): columns past E load the last ones, and
// `keep` puts -inf there and everywhere in a row that does not count, whatever it holds.
template <int G, int NV, int W>
MOE_DEV void load_row(const float* row, int E, int q, float (&v)[NV * W]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = min(W * (i * G + q), E - W);
    if constexpr (W == 4) {
      const float4 f = *(const float4*)(row + e);
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    } else {
      v[i] = row[e];
    }
  }
}
template <int G, int NV, int W>
MOE_DEV void keep(float (&v)[NV * W], int E, int q, bool counted) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int w = 0; w < W; ++w)
      v[i * W + w] = counted && W * (i * G + q) < E ? v[i * W + w] : -__builtin_huge_valf();
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
  // U rows of a group are loaded together (a short input is bound by the latency of its loads), and the next U while
  // these are summed. Every lane runs the same trip count, so the reductions are never divergent.
  constexpr int U = G >= 32 ? 4 : G / 8;  // (with 8 lanes a row, one pass is the smallest tile)
  const uint8_t* const mk = mask ? mask : (const uint8_t*)logits;  // no mask: any readable byte, not looked at
  struct Rows { float v[U][C]; int k[U]; uint8_t m[U]; };
  auto load = [&](Rows& b, int64_t rb) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = min(rb + u * RP + g, t.r1 - 1);
      load_row<G, NV, W>(logits + r * E, E, q, b.v[u]);
      b.m[u] = mk[r];
      b.k[u] = idx[r * K + min(q, K - 1)];
    }
  };
  Rows next;
  load(next, t.r0);
  for (int64_t rb = t.r0; rb < t.r1; rb += RP * U) {
    Rows cur = next;
    if (rb + RP * U < t.r1) load(next, rb + RP * U);
    float (&v)[U][C] = cur.v;
    int my[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool counted = rb + u * RP + g < t.r1 && (!mask || cur.m[u] != 0);
      keep<G, NV, W>(v[u], E, q, counted);
      my[u] = counted && q < K ? cur.k[u] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = rb + u * RP + g;
      float m = v[u][0];
#pragma unroll
      for (int c = 1; c < C; ++c) m = fmaxf(m, v[u][c]);
      m = group_max<G>(m);
      if (m == -__builtin_huge_valf()) m = 0.f;  // no finite logit: the sum below is 0, or NaN
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        v[u][c] = __expf(v[u][c] - m);
        s += v[u][c];
      }
      s = group_sum<G>(s);
      const bool live = s != 0.f;  // a row of -inf only is left out like a masked one
      const float lse = live ? m + __logf(s) : 0.f;
      const float inv = live ? 1.0f / s : 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = fmaf(v[u][c], inv, acc[c]);
      z = fma((double)lse, (double)lse, z);
      n += live ? 1 : 0;
      if (r < t.r1 && q == 0) lse_out[r] = lse;
      if (live && my[u] >= 0 && my[u] < E) atomicAdd(&hist[my[u]], 1);
    }
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

template <class T>
MOE_DEV void st_device(T* p, T v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <class T>
MOE_DEV T ld_device(T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Sums over the wave's lanes of equal lane % W.
template <int W>
MOE_DEV double lanes_sum(double v) {
#pragma unroll
  for (int o = 32; o >= W; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}
template <int W>
MOE_DEV int lanes_sum(int v) {
#pragma unroll
  for (int o = 32; o >= W; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// Adds the tiles of each segment in a fixed order: one block of RT threads per segment and RC columns, RT / RC
// tiles side by side, one barrier. The last block to arrive forms the losses from the segments' sums. 1024
// threads on 16 columns (64 tiles at once), or, for segments of a few tiles, 256 on 32: fewer lanes
// without a tile and half the arrivals (267 tokens of 212 experts in 57 segments, with their gradient, 26 -> 20 us,
// 11973 of 184 in 63 29 -> 23 us; one wide segment of 1000 tiles 10 us of its own).
template <int RT, int RC>
__global__ __launch_bounds__(RT) void router_loss_reduce_kernel(
    Pieces pc, LossWs ws, int64_t slots, int E, int K, float balance_coef, float z_coef, int32_t* __restrict__ seg_counts,
    int32_t* __restrict__ seg_tokens, float* __restrict__ seg_probs, float* __restrict__ loss) {
  constexpr int NW = RT / kWave;
  __shared__ double red[NW][RC + 1];
  __shared__ int redc[NW][RC + 1];
  __shared__ bool last;
  const int nb = (E + RC - 1) / RC;
  const int s = blockIdx.x / nb, cb = blockIdx.x % nb;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = tid % RC, grp = tid / RC;
  const int e = cb * RC + col;
  const int64_t b0 = pc.bound(s + 1), b1 = pc.bound(s + 2);
  const int64_t first = (b0 >> pc.shift) + s + 1;
  int64_t end = b1 > b0 ? first + ((b1 - b0 + pc.R - 1) >> pc.shift) : first;
  if (end > slots) end = slots;

  double p = 0.0, z = 0.0;
  int c = 0, n = 0;
  if (e < E)
#pragma unroll 8
    for (int64_t i = first + grp; i < end; i += (RT / RC)) {
      p += (double)ws.p[i * E + e];
      c += ws.c[i * E + e];
    }
  if (cb == 0)
    for (int64_t i = first + tid; i < end; i += RT) { z += ws.z[i]; n += ws.n[i]; }
  p = lanes_sum<RC>(p);
  c = lanes_sum<RC>(c);
  if (lane < RC) { red[wave][lane] = p; redc[wave][lane] = c; }
  if (cb == 0) {
    z = lanes_sum<1>(z);
    n = lanes_sum<1>(n);
    if (lane == 0) { red[wave][RC] = z; redc[wave][RC] = n; }
  }
  __syncthreads();
  if (wave == 0) {
    p = 0.0;
    c = 0;
    if (lane < RC || (cb == 0 && lane == RC))
#pragma unroll
      for (int w = 0; w < NW; ++w) { p += red[w][lane]; c += redc[w][lane]; }
    if (lane < RC && e < E) {
      seg_probs[(int64_t)s * E + e] = (float)p;
      seg_counts[(int64_t)s * E + e] = c;
    }
    const double cp = lanes_sum<1>(lane < RC && e < E ? p * (double)c : 0.0);
    // What the last block reads is stored and loaded past the XCD's L2 (device-scope atomics), so the
    // stores need only be complete before the arrival: a fence would write the whole L2 back.
    if (lane == 0) st_device(&ws.cp[(int64_t)s * nb + cb], cp);
    if (cb == 0 && lane == RC) { st_device(&ws.zs[s], p); st_device(&seg_tokens[s], c); }
    asm volatile("" ::: "memory");
    wait_vm<0>();
    asm volatile("" ::: "memory");
    if (lane == 0) last = atomicAdd(ws.arrived, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  double bal = 0.0;
  z = 0.0;
  n = 0;
  int full = 0;
  for (int i = tid; i < pc.S; i += RT) {
    const int ns = ld_device(&seg_tokens[i]);
    const double zs = ld_device(&ws.zs[i]);  // an empty segment's sums are zeros
    double cp = 0.0;
#pragma unroll 8
    for (int j = 0; j < nb; ++j) cp += ld_device(&ws.cp[(int64_t)i * nb + j]);
    bal += ns > 0 ? cp * (double)E / ((double)ns * (double)ns * (double)K) : 0.0;
    z += zs;
    n += ns;
    full += ns > 0 ? 1 : 0;
  }
  bal = lanes_sum<1>(bal);
  z = lanes_sum<1>(z);
  n = lanes_sum<1>(n);
  full = lanes_sum<1>(full);
  if (lane == 0) { red[wave][0] = bal; red[wave][1] = z; redc[wave][0] = n; redc[wave][1] = full; }
  __syncthreads();
  if (tid == 0) {
    bal = z = 0.0;
    n = full = 0;
    for (int w = 0; w < NW; ++w) { bal += red[w][0]; z += red[w][1]; n += redc[w][0]; full += redc[w][1]; }
    const double lb = full ? bal / full : 0.0, lz = n ? z / n : 0.0;
    // a z part that is not used stays out: it may be infinite
    loss[0] = (float)((double)balance_coef * lb + (z_coef != 0.f ? (double)z_coef * lz : 0.0));
    loss[1] = (float)lb;
    loss[2] = (float)lz;
    seg_tokens[pc.S] = n;
    seg_tokens[pc.S + 1] = full;
    *ws.arrived = 0;
  }
}

// One segment of few tiles: one block adds them all, columns side by side in `ec` threads (E rounded up to a
// power of two), and forms the losses with no exchange between blocks (512 tokens 4.4 us, 7 us with it).
__global__ __launch_bounds__(kRedThreads) void router_loss_reduce_one_kernel(
    Pieces pc, LossWs ws, int64_t slots, int E, int K, int ec, float balance_coef, float z_coef,
    int32_t* __restrict__ seg_counts, int32_t* __restrict__ seg_tokens, float* __restrict__ seg_probs,
    float* __restrict__ loss) {
  constexpr int NW = kRedThreads / kWave;
  __shared__ double redp[kRedThreads], red[NW], redz[NW];
  __shared__ int redc[kRedThreads], redn[NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = tid & (ec - 1), grp = tid / ec, groups = kRedThreads / ec;
  const int64_t b0 = pc.bound(1), b1 = pc.bound(2), first = (b0 >> pc.shift) + 1;
  int64_t end = b1 > b0 ? first + ((b1 - b0 + pc.R - 1) >> pc.shift) : first;
  if (end > slots) end = slots;
  double p = 0.0, z = 0.0;
  int c = 0, n = 0;
  if (col < E)
#pragma unroll 8
    for (int64_t i = first + grp; i < end; i += groups) {
      p += (double)ws.p[i * E + col];
      c += ws.c[i * E + col];
    }
  for (int64_t i = first + tid; i < end; i += kRedThreads) { z += ws.z[i]; n += ws.n[i]; }
  redp[tid] = p;
  redc[tid] = c;
  z = lanes_sum<1>(z);
  n = lanes_sum<1>(n);
  if (lane == 0) { redz[wave] = z; redn[wave] = n; }
  __syncthreads();
  double cp = 0.0;
  if (tid < E) {
    for (int k = 1; k < groups; ++k) { p += redp[k * ec + tid]; c += redc[k * ec + tid]; }
    seg_probs[tid] = (float)p;
    seg_counts[tid] = c;
    cp = p * (double)c;
  }
  cp = lanes_sum<1>(cp);
  if (lane == 0) red[wave] = cp;
  __syncthreads();
  if (tid == 0) {
    cp = z = 0.0;
    n = 0;
    for (int w = 0; w < NW; ++w) { cp += red[w]; z += redz[w]; n += redn[w]; }
    const double lb = n ? cp * (double)E / ((double)n * (double)n * (double)K) : 0.0, lz = n ? z / n : 0.0;
    loss[0] = (float)((double)balance_coef * lb + (z_coef != 0.f ? (double)z_coef * lz : 0.0));
    loss[1] = (float)lb;
    loss[2] = (float)lz;
    seg_tokens[0] = n;
    seg_tokens[1] = n;
    seg_tokens[2] = n > 0 ? 1 : 0;
  }
}

// Several segments of few tiles: one block loads all their partials into LDS at once and adds each segment's in tile
// order (12 tokens in 22 segments 4.8 us, 7 us with the exchange between blocks; in the forward's last block, which
// has to wait for the others' stores, 6 us). One segment by the kernel above is 0.5 us faster than here.
constexpr size_t kSmallLds = 30 * 1024;  // (more takes as long here as with the exchange)
struct SmallSlot { double z; int n, first, end; };  // a tile's sums; the tiles of segment i (there are more tiles than segments)
static size_t small_lds(int64_t slots, int E) { return (size_t)(slots * (sizeof(SmallSlot) + 8 * (int64_t)E)); }

__global__ __launch_bounds__(kRedThreads) void router_loss_reduce_small_kernel(
    Pieces pc, LossWs ws, int slots, int E, int K, float balance_coef, float z_coef, int32_t* __restrict__ seg_counts,
    int32_t* __restrict__ seg_tokens, float* __restrict__ seg_probs, float* __restrict__ loss) {
  constexpr int NW = kRedThreads / kWave;
  extern __shared__ SmallSlot slot[];
  float* const pp = (float*)(slot + slots);
  int* const cc = (int*)(pp + slots * E);
  __shared__ double red[2][NW];
  __shared__ int redc[2][NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (wave == 0) {  // side by side with the other waves' loads
    for (int i = lane; i < slots; i += kWave) {
      slot[i].z = ws.z[i];
      slot[i].n = ws.n[i];
      if (i >= pc.S) continue;
      const int64_t b0 = pc.bound(i + 1), b1 = pc.bound(i + 2);
      slot[i].first = (int)((b0 >> pc.shift) + i + 1);
      slot[i].end = min(slots, slot[i].first + (b1 > b0 ? (int)((b1 - b0 + pc.R - 1) >> pc.shift) : 0));
    }
  } else {
#pragma unroll 4
    for (int i = tid - kWave; i < slots * E; i += kRedThreads - kWave) { pp[i] = ws.p[i]; cc[i] = ws.c[i]; }
  }
  __syncthreads();
  double bal = 0.0, z = 0.0;
  int n = 0, full = 0;
  for (int i = tid; i < pc.S * E; i += kRedThreads) {
    const int s = i / E, e = i % E;
    const int first = slot[s].first, end = slot[s].end;
    double p = 0.0;
    int c = 0, ns = 0;
#pragma unroll 4
    for (int j = first; j < end; ++j) {
      p += (double)pp[j * E + e];
      c += cc[j * E + e];
      ns += slot[j].n;
    }
    seg_probs[i] = (float)p;
    seg_counts[i] = c;
    if (ns > 0) bal += p * (double)c * (double)E / ((double)ns * (double)ns * (double)K);
    if (e == 0) {
      seg_tokens[s] = ns;
      for (int j = first; j < end; ++j) z += slot[j].z;
      n += ns;
      full += ns > 0 ? 1 : 0;
    }
  }
  bal = lanes_sum<1>(bal);
  z = lanes_sum<1>(z);
  n = lanes_sum<1>(n);
  full = lanes_sum<1>(full);
  if (lane == 0) { red[0][wave] = bal; red[1][wave] = z; redc[0][wave] = n; redc[1][wave] = full; }
  __syncthreads();
  if (tid == 0) {
    bal = z = 0.0;
    n = full = 0;
    for (int w = 0; w < NW; ++w) { bal += red[0][w]; z += red[1][w]; n += redc[0][w]; full += redc[1][w]; }
    const double lb = full ? bal / full : 0.0, lz = n ? z / n : 0.0;
    loss[0] = (float)((double)balance_coef * lb + (z_coef != 0.f ? (double)z_coef * lz : 0.0));
    loss[1] = (float)lb;
    loss[2] = (float)lz;
    seg_tokens[pc.S] = n;
    seg_tokens[pc.S + 1] = full;
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
  const double even = (double)ns * K;  // slots of the segment (whole numbers below 2^53: exact)
  const float per = ns > 0 && full > 0 ? balance_coef / ((float)full * (float)ns * (float)even) : 0.f;
  const float zc = N > 0 ? 2.f * z_coef / (float)N : 0.f;
  const float gl = dloss ? *dloss : 1.f;
  constexpr int U = 4;
  const uint8_t* const mk = mask ? mask : (const uint8_t*)logits;  // no mask: any readable byte, not looked at
  struct Rows { float v[U][C], lse[U]; uint8_t m[U]; };
  auto load = [&](Rows& b, int64_t rb) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = min(rb + u * RP + g, t.r1 - 1);
      load_row<G, NV, W>(logits + r * E, E, q, b.v[u]);
      b.lse[u] = lse_in[r];
      b.m[u] = mk[r];
    }
  };
  Rows next;
  load(next, t.r0);
  float w[C];
  bool have_w = false;
  for (int64_t rb = t.r0; rb < t.r1; rb += RP * U) {
    Rows cur = next;
    if (rb + RP * U < t.r1) load(next, rb + RP * U);
    float (&v)[U][C] = cur.v, (&lse)[U] = cur.lse;
    bool counted[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      counted[u] = rb + u * RP + g < t.r1 && !outside && (!mask || cur.m[u] != 0);
      keep<G, NV, W>(v[u], E, q, counted[u]);
      lse[u] = counted[u] ? lse[u] : 0.f;
    }
    if (!have_w) {  // the segment's coefficients, behind the first rows' loads
      have_w = true;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const int e = W * (i * G + q) + j;
          w[i * W + j] = ns > 0 && e < E ? per * (float)((double)seg_counts[(int64_t)s * E + e] * E - even) : 0.f;
        }
    }
    // lse keeps only the digits that its size leaves, up to log E is lost where the logits are huge,
    // so the probabilities are normalised again (the exponent stays within log E of the true one)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = rb + u * RP + g;
      float d = 0.f, sum = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        v[u][c] = __expf(v[u][c] - lse[u]);
        sum += v[u][c];
        d = fmaf(v[u][c], w[c], d);
      }
      sum = group_sum<G>(sum);
      d = group_sum<G>(d);
      if (r >= t.r1) continue;
      // no finite logit: left out like a masked row, with zeros whatever dloss and the coefficients are
      const bool live = counted[u] && sum != 0.f;
      const float inv = live ? 1.0f / sum : 0.f;
      const float add = zc * lse[u] - d * inv, scale = gl * inv;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = W * (i * G + q);
        if (e >= E) continue;
        float o[W];
#pragma unroll
        for (int j = 0; j < W; ++j) o[j] = live ? scale * v[u][i * W + j] * (w[i * W + j] + add) : 0.f;
        // (whole lines past the L2: 40000 tokens of 160 experts with the forward 33 -> 30 us, 131072 of 256 84 -> 80.5)
        if constexpr (W == 4) __builtin_nontemporal_store(f32x4_t{o[0], o[1], o[2], o[3]}, (f32x4_t*)(dlogits + r * E + e));
        else dlogits[r * E + e] = o[0];
      }
    }
  }
}

// Lanes per row and registers per lane by E; rows that are not whole aligned 16-byte vectors go by single values.
// Forward: four vectors a lane where they fill them (two up to 64 experts), so that the steps of a row's
// reductions serve more rows at once (35K tokens of 96 experts 10 us with one vector a lane, 7 us so).
// Backward: one or two, because every lane forms the coefficients of its own columns first (512 tokens
// of 128 experts 7.4 us with four vectors a lane, 5.3 us so).
#define MOE_LOSS_SHAPE(E, vec, FWD, ...)                                                        \
  do {                                                                                          \
    if (vec) {                                                                                  \
      if ((E) <= 64) { constexpr int G = FWD ? 8 : 16, NV = FWD ? 2 : 1, W = 4; __VA_ARGS__; }   \
      else if ((E) <= 128) { constexpr int G = FWD ? 8 : 32, NV = FWD ? 4 : 1, W = 4; __VA_ARGS__; }  \
      else if ((E) <= 256) { constexpr int G = FWD ? 16 : 32, NV = FWD ? 4 : 2, W = 4; __VA_ARGS__; } \
      else if ((E) <= 512) { constexpr int G = FWD ? 32 : 64, NV = FWD ? 4 : 2, W = 4; __VA_ARGS__; } \
      else { constexpr int G = 64, NV = 4, W = 4; __VA_ARGS__; }                                \
    } else if ((E) <= 128) { constexpr int G = 64, NV = 2, W = 1; __VA_ARGS__; }                \
    else { constexpr int G = 64, NV = 16, W = 1; __VA_ARGS__; }                                 \
  } while (0)

hipError_t launch_router_loss(const float* logits, const int32_t* topk_idx, const int32_t* seg_offsets,
                              const uint8_t* mask, float* lse, int32_t* seg_counts, int32_t* seg_tokens,
                              float* seg_probs, float* loss, void* workspace, int64_t T, int E, int K, int S,
                              float balance_coef, float z_coef, hipStream_t s) {
  const LossWs ws = loss_ws(workspace, T, S, E, nullptr);
  const int R = router_loss_tile(T);
  const Pieces pc{seg_offsets, T, S, R, __builtin_ctz(R)};
  const int64_t slots = loss_slots(T, S);
  if (T > 0) {
    const bool vec = E % 4 == 0 && (uintptr_t)logits % 16 == 0;
    MOE_TRACE("router_loss_stats", s);
    MOE_LOSS_SHAPE(E, vec, true, MOE_LAUNCH((router_loss_stats_kernel<G, NV, W>), dim3((unsigned)slots), dim3(kLossThreads), 0, s,
                                      logits, topk_idx, mask, lse, pc, ws, E, K));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (S == 1 && slots <= 70) {  // at most 64 tiles of 32 rows and the pieces' edges
    int ec = 64;
    while (ec < E) ec *= 2;
    MOE_TRACE("router_loss_reduce", s);
    MOE_LAUNCH(router_loss_reduce_one_kernel, dim3(1), dim3(kRedThreads), 0, s, pc, ws, slots, E, K, ec, balance_coef, z_coef,
               seg_counts, seg_tokens, seg_probs, loss);
  } else if (S > 1 && slots <= 4096 && small_lds(slots, E) <= kSmallLds) {
    MOE_TRACE("router_loss_reduce", s);
    MOE_LAUNCH(router_loss_reduce_small_kernel, dim3(1), dim3(kRedThreads), small_lds(slots, E), s, pc, ws, (int)slots, E, K,
               balance_coef, z_coef, seg_counts, seg_tokens, seg_probs, loss);
  } else {
    MOE_TRACE("router_loss_reduce", s);
    const bool narrow = slots <= 30 * (int64_t)S;
    const int rc = narrow ? 2 * kRedCols : kRedCols, rt = narrow ? 256 : kRedThreads;
    MOE_LAUNCH(narrow ? (router_loss_reduce_kernel<256, 2 * kRedCols>) : (router_loss_reduce_kernel<kRedThreads, kRedCols>),
               dim3((unsigned)((int64_t)S * ((E + rc - 1) / rc))), dim3(rt), 0, s, pc, ws, slots, E, K, balance_coef, z_coef,
               seg_counts, seg_tokens, seg_probs, loss);
  }
  return hipGetLastError();
}

hipError_t launch_router_loss_bwd(const float* logits, const float* lse, const int32_t* seg_offsets,
                                  const uint8_t* mask, const int32_t* seg_counts, const int32_t* seg_tokens,
                                  const float* dloss, float* dlogits, int64_t T, int E, int K, int S,
                                  float balance_coef, float z_coef, hipStream_t s) {
  if (T <= 0) return hipSuccess;
  const int R = router_loss_tile(T);
  const Pieces pc{seg_offsets, T, S, R, __builtin_ctz(R)};
  const bool vec = E % 4 == 0 && (uintptr_t)logits % 16 == 0 && (uintptr_t)dlogits % 16 == 0;
  {
    MOE_TRACE("router_loss_bwd", s);
    MOE_LOSS_SHAPE(E, vec, false, MOE_LAUNCH((router_loss_bwd_kernel<G, NV, W>), dim3((unsigned)loss_slots(T, S)),
                                      dim3(kLossThreads), 0, s, logits, lse, mask, seg_counts, seg_tokens, dloss, dlogits,
                                      pc, E, K, balance_coef, z_coef));
  }
  return hipGetLastError();
}

}  // namespace moe
