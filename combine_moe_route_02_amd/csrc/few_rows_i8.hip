// 8-bit integer expert products for a few rows per expert (decode batches): the weights of every expert
// that has rows are streamed once and everything else is small, so the time is the weights' bytes.
//
// The grouped GEMM's smallest tiles (64 x 64) walk K pair by pair at 0.3 us however few rows they hold, a few experts
// fill few CUs with them, and h takes a launch of its own to be quantised. These kernels give 16, 32 or 64 columns of one
// expert to a workgroup of four waves. A wave loads the weights of its 16 columns straight into registers as
// v_mfma_i32_16x16x64_i8 operands (16 columns x 64 bytes, no LDS: no weight is used by two waves), one
// batch of K steps ahead. With 64 columns each wave runs the whole of K; with fewer, 2 or 4 waves share
// the columns and take the K steps in turn, so that a few experts still fill the CUs, and their int32
// sums meet in LDS. The sums are exact: neither the split nor the choice between these kernels and the
// GEMM's changes a bit of the result.
//
// The rows' operand comes from L2 the same way (staging it in LDS for the four waves measured slower: a
// barrier and a load latency per chunk of K; 32 rows x 7168 on 4096 columns 33 against 19 us). Only down
// stages: gate/up leaves h in FP32 with the largest magnitude of every row and 16-column slice (in the
// codes half of the h buffer, unused here), and down forms each row's scale from them and quantises h
// once per workgroup, with the FP32 steps of the quantisation kernels.
//
// Both products and h's codes, H = 2048, I = 768, 128 experts, top-8 (here / GEMM path, us): 1 token 15 / 23, 4 tokens 29 /
// 40, 16 tokens 93 / 104, 33 tokens 115 / 122. A pass holds the rows that even routing gives an expert; one with many more takes
// its weights through again for every pass (the figures of uneven routing stand at few_rows_layer).
// The same layer: one token (8 experts, 38 MB of weights) 9 us gate/up and 7 us down, of which a
// launch's first loads and the sums' exchange are half; 33 tokens (all but a few experts) 72 and 47 us, 4.8 and 3.8
// TB/s. Twice the loads in flight are slower (16 rows x 7168 on 4096 columns 10.5 -> 11.0 us, 32 rows 12.5 -> 15).
#include <algorithm>
#include <cmath>

#include "common.h"
#include "i8.h"
#include "launch.h"
#include "trace.h"

namespace moe {
namespace {

constexpr int kFewThreads = 256, kFewWaves = 4;
constexpr int kCols = 16;     // columns of a weight operand
constexpr int kMaxRows = 128;  // rows of one pass over the weights

// Staging (down): 16 NB rows of up to chunk_k bytes of K, each with 16 bytes of padding (a fragment read of
// 16 rows then touches all banks evenly).
template <int NB> constexpr int chunk_k() { return NB <= 2 ? 2048 : NB <= 4 ? 1024 : 512; }
constexpr int kScaleBytes = kMaxRows * 8;  // multiplier and scale per row
MOE_DEV int pitch_k(int K, int chunk) { return min(K, chunk) + 16; }

enum FewMode { kFewGateUp = 0, kFewCodes = 1, kFewDown = 2 };

struct FewArgs {
  const int8_t* x;          // kFewGateUp, kFewCodes: [P, K] codes
  const float* x_scale;     // [P]
  const float* h;           // kFewDown: [P, K] FP32 rows (gate/up writes them: out_h)
  uint32_t* part;           // [P, K / 4] words: the row's largest magnitude in slice i is word i
  const int8_t* w;          // per group [N, K] (gate/up: [2 N, K], gate rows first)
  const float* w_scale;     // per group [N] ([2 N])
  float* out_h;             // kFewGateUp: [P, N]
  uint16_t* y;              // kFewCodes: [P, N] BF16; kFewDown: rows of yd (i8.h)
  const int32_t* offsets;   // null: one group of P_c rows
  int64_t P_c;
  int K, N, El, c0, groups; // groups = El * chunks
  int ctiles;
  bool listed;              // block / ctiles counts the groups that have rows, else it is the group
};

MOE_DEV void group_rows(const FewArgs& a, int g, int64_t& r0, int& n) {
  if (!a.offsets) { r0 = 0; n = (int)a.P_c; return; }
  const int c = a.c0 + g / a.El, e = g % a.El;
  const int32_t* off = a.offsets + (int64_t)c * (a.El + 1);
  const int o0 = max(0, min(off[e], (int)a.P_c)), o1 = max(o0, min(off[e + 1], (int)a.P_c));
  r0 = (int64_t)c * a.P_c + o0;
  n = o1 - o0;
}

// The group of this workgroup and its rows; -1 if there is none. Every thread calls it.
MOE_DEV int find_group(const FewArgs& a, int want, int64_t& r0, int& n) {
  if (!a.listed) {
    group_rows(a, want, r0, n);
    return want;
  }
  __shared__ int cnt[kFewWaves], found[2];
  __shared__ int64_t start;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) found[0] = -1;
  int before = 0;
  for (int g0 = 0; g0 < a.groups; g0 += kFewThreads) {
    const int g = g0 + tid;
    int64_t r = 0;
    int len = 0;
    if (g < a.groups) group_rows(a, g, r, len);
    const uint64_t m = __ballot(len > 0);
    if (lane == 0) cnt[wave] = __popcll(m);
    __syncthreads();
    int at = before;
    for (int i = 0; i < kFewWaves; ++i) {
      if (i < wave) at += cnt[i];
      before += cnt[i];
    }
    if (len > 0 && at + __popcll(m & ((1ull << lane) - 1)) == want) { found[0] = g; found[1] = len; start = r; }
    __syncthreads();
    if (before > want) break;
  }
  const uint64_t r = start;
  r0 = ((int64_t)__builtin_amdgcn_readfirstlane((int)(r >> 32)) << 32) | (uint32_t)__builtin_amdgcn_readfirstlane((int)r);
  n = __builtin_amdgcn_readfirstlane(found[1]);
  return __builtin_amdgcn_readfirstlane(found[0]);
}

// Stage the codes of K values [k0, k0 + kc) of the pass's rows, 16 FP32 values to a 16-byte piece. Rows past
// the pass's last one are left as they are: their products are not stored.
template <int NB>
MOE_DEV void stage_rows(const FewArgs& a, int64_t r0, int m0, int n, int k0, int kc, char* xs, const float* scales) {
  const int pieces = kc / 16, total = (n - m0) * pieces, pitch = pitch_k(a.K, chunk_k<NB>());
  constexpr int B = 2;  // pieces of a thread in flight
  for (int i0 = threadIdx.x; i0 < total; i0 += B * kFewThreads) {
    float4 f[B][4];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int i = min(i0 + u * kFewThreads, total - 1), r = m0 + i / pieces;
      const float4* p = (const float4*)(a.h + (r0 + r) * a.K + k0 + 16 * (i % pieces));
#pragma unroll
      for (int j = 0; j < 4; ++j) f[u][j] = p[j];
    }
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int i = i0 + u * kFewThreads;
      if (i >= total) continue;
      const int r = i / pieces;
      const float inv = scales[2 * r];
      uint4 c;
      c.x = codes4(f[u][0].x, f[u][0].y, f[u][0].z, f[u][0].w, inv);
      c.y = codes4(f[u][1].x, f[u][1].y, f[u][1].z, f[u][1].w, inv);
      c.z = codes4(f[u][2].x, f[u][2].y, f[u][2].z, f[u][2].w, inv);
      c.w = codes4(f[u][3].x, f[u][3].y, f[u][3].z, f[u][3].w, inv);
      *(uint4*)(xs + r * pitch + 16 * (i % pieces)) = c;
    }
  }
}

// The scale of each row of a pass from the largest magnitudes of its slices, 16 lanes per row.
MOE_DEV void row_scales(const FewArgs& a, int64_t r0, int m0, int n, float* scales) {
  const int tid = threadIdx.x, parts = a.K / kCols;
  for (int i = tid >> 4; i < n - m0; i += kFewThreads / 16) {
    const uint32_t* p = a.part + (r0 + m0 + i) * (a.K / 4);
    uint32_t big = 0;
    for (int s = tid & 15; s < parts; s += 16) big = max(big, p[s]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, o, kWave));
    const RowScale q = row_scale(big);
    if ((tid & 15) == 0) {
      scales[2 * i] = q.inv;
      scales[2 * i + 1] = q.scale;
    }
  }
}

// One pass: rows m0 .. n - 1 of the group at r0 (at most 16 NB), columns n0 .. of the workgroup.
// CB: weight operands of a wave (gate and up of 16 columns, or 16 or 32 columns).
template <int MODE, int NB, int KW, int CB>
MOE_DEV void few_pass(const FewArgs& a, int e, int64_t r0, int m0, int n, int n0, char* lds) {
  constexpr bool kStaged = MODE == kFewDown, kGU = MODE == kFewGateUp;
  constexpr int CW = kFewWaves / KW;              // waves side by side in columns
  constexpr int CS = chunk_k<NB>() / 64;          // K steps of a staged chunk
  // K steps of a batch (two in flight): about 16 KiB of weights and rows a wave
  constexpr int UM = kStaged ? 8 / CB : NB == 1 ? 8 / CB : NB == 2 ? 4 : NB <= 4 ? 2 : 1;
  constexpr int U = kStaged && CS / KW < UM ? CS / KW : UM;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cw = wave % CW, kw = wave / CW;
  const int lr = lane & 15, lk = 16 * (lane >> 4);
  const int col0 = n0 + (kGU ? kCols : kCols * CB) * cw;
  float* const scales = (float*)lds;
  char* const xs = lds + kScaleBytes;
  const int8_t* wp[CB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)  // columns past N read the last one; they are not stored
    wp[cb] = a.w + (kGU ? (int64_t)e * (2 * a.N) + (int64_t)cb * a.N + min(col0 + lr, a.N - 1)
                        : (int64_t)e * a.N + min(col0 + kCols * cb + lr, a.N - 1)) * a.K + lk;
  const int8_t* xp[NB];
  if constexpr (!kStaged)
#pragma unroll
    for (int b = 0; b < NB; ++b)  // rows past the last one read it; they are not stored
      xp[b] = a.x + (r0 + min(m0 + 16 * b + lr, n - 1)) * a.K + lk;
  const int ns = a.K / 64;  // K steps
  // The wave's t-th step: pairs of steps (whole 128-byte lines of a row) go round the KW waves.
  auto step_of = [&](int t) { return 2 * ((t >> 1) * KW + kw) + (t & 1); };
  struct Batch { i32x4_t w[U][CB], x[kStaged ? 1 : U][NB]; };
  auto load = [&](Batch& d, int t) {  // steps past the end read the last one; they are not used
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = 64 * min(step_of(t + u), ns - 1);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) d.w[u][cb] = *(const i32x4_t*)(wp[cb] + at);
      if constexpr (!kStaged)
#pragma unroll
        for (int b = 0; b < NB; ++b) d.x[u][b] = *(const i32x4_t*)(xp[b] + at);
    }
  };
  Batch cur, next;
  load(cur, 0);
  if (step_of(U) < ns) load(next, U);
  // what the end needs, behind the first weights
  const int c = col0 + 4 * (lane >> 4);  // N is a multiple of 8: four columns end together
  float sb[CB][4], sr[NB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      sb[cb][q] = kGU ? a.w_scale[(int64_t)e * (2 * a.N) + (int64_t)cb * a.N + min(c, a.N - 4) + q]
                      : a.w_scale[(int64_t)e * a.N + min(c + kCols * cb, a.N - 4) + q];
  if constexpr (kStaged) {
    row_scales(a, r0, m0, n, scales);
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b) sr[b] = a.x_scale[r0 + min(m0 + 16 * b + lr, n - 1)];
  }
  i32x4_t acc[CB][NB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[cb][b] = i32x4_t{0, 0, 0, 0};
  // the batch at the wave's step t, then the one after next on its way
  auto batch = [&](int t, int end, auto&& operand) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (step_of(t + u) < end) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const i32x4_t x = operand(u, b, step_of(t + u));
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) acc[cb][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(cur.w[u][cb], x, acc[cb][b], 0, 0, 0);
        }
      }
    cur = next;
    if (step_of(t + 2 * U) < ns) load(next, t + 2 * U);
  };
  if constexpr (kStaged) {
    const int pitch = pitch_k(a.K, chunk_k<NB>());
    for (int s0 = 0; s0 < ns; s0 += CS) {
      __syncthreads();  // the chunk before this one has been read
      stage_rows<NB>(a, r0, m0, n, 64 * s0, 64 * min(CS, ns - s0), xs, scales);
      __syncthreads();
      const char* p = xs + lr * pitch + lk;
      const int end = min(s0 + CS, ns);
      for (int t = s0 / KW; t < (s0 + CS) / KW && step_of(t) < end; t += U)
        batch(t, end, [&](int, int b, int at) { return *(const i32x4_t*)(p + 16 * b * pitch + 64 * (at - s0)); });
    }
  } else {
    for (int t = 0; step_of(t) < ns; t += U) batch(t, ns, [&](int u, int b, int) { return cur.x[u][b]; });
  }
  // lane: row lane & 15 of a block, columns 4 (lane >> 4) .. + 3
  auto finish = [&](int b, float srow, const i32x4_t (&v)[CB]) {
    const int m = m0 + 16 * b + lr;
    const int64_t row = r0 + min(m, n - 1);
    if constexpr (MODE == kFewDown) srow = scales[2 * (min(m, n - 1) - m0) + 1];
    float o[4];
    if constexpr (MODE == kFewGateUp) {
      uint32_t big = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float gf = (float)v[0][q] * (srow * sb[0][q]), uf = (float)v[1][q] * (srow * sb[1][q]);
        o[q] = gf * sigmoidf_(gf) * uf;
        big = max(big, __float_as_uint(o[q]) & 0x7fffffffu);
      }
      big = max(big, (uint32_t)__shfl_xor((int)big, 16, kWave));
      big = max(big, (uint32_t)__shfl_xor((int)big, 32, kWave));
      if (m < n && c < a.N) *(float4*)(a.out_h + row * a.N + c) = make_float4(o[0], o[1], o[2], o[3]);
      if (m < n && col0 < a.N && lane < 16) a.part[row * (a.N / 4) + col0 / kCols] = big;
    } else {
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = (MODE == kFewDown ? kYdUnit * (float)v[cb][q] : (float)v[cb][q]) * (srow * sb[cb][q]);
        const int at = c + kCols * cb;
        const uint2 p = MODE == kFewDown ? make_uint2(pack_yd(o[0], o[1]), pack_yd(o[2], o[3]))
                                         : make_uint2(pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3]));
        if (m < n && at < a.N) *(uint2*)(a.y + row * a.N + at) = p;
      }
    }
  };
  if constexpr (KW == 1) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      i32x4_t v[CB];
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) v[cb] = acc[cb][b];
      finish(b, sr[b], v);
    }
  } else {
    i32x4_t* red = (i32x4_t*)xs;  // [KW][CW][CB][NB][64]: at most 64 KiB
    __syncthreads();
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int b = 0; b < NB; ++b) red[((wave * CB + cb) * NB + b) * 64 + lane] = acc[cb][b];
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b % KW != kw) continue;
      i32x4_t v[CB];
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        v[cb] = red[((cw * CB + cb) * NB + b) * 64 + lane];
#pragma unroll
        for (int k = 1; k < KW; ++k) v[cb] += red[(((k * CW + cw) * CB + cb) * NB + b) * 64 + lane];
      }
      finish(b, sr[b], v);
    }
  }
}

// Weight operands of a wave, and columns of a workgroup. WIDE: a wave of the plain product or of down takes 32
// columns, so that each load of rows serves two operands. NBM: blocks of 16 rows that a pass holds at most.
template <int MODE, bool WIDE> constexpr int wave_operands() { return MODE == kFewGateUp || WIDE ? 2 : 1; }
template <int KW, bool WIDE> constexpr int wg_cols() { return (WIDE ? 2 : 1) * kCols * kFewWaves / KW; }

template <int MODE, int KW, int NBM, bool WIDE>
__global__ __launch_bounds__(kFewThreads) void few_rows_i8_kernel(FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int CB = wave_operands<MODE, WIDE>();
  int64_t r0;
  int n;
  const int g = find_group(a, blockIdx.x / a.ctiles, r0, n), n0 = (blockIdx.x % a.ctiles) * wg_cols<KW, WIDE>();
  if (g < 0) return;
  const int e = g % a.El;
  for (int m0 = 0; m0 < n; m0 += 16 * NBM) {
    const int left = min(n - m0, 16 * NBM);
    if (m0 > 0) __syncthreads();  // the last rows' scales and sums have been read
#define MOE_FEW(NB_) few_pass<MODE, (NB_ < NBM ? NB_ : NBM), KW, CB>(a, e, r0, m0, m0 + left, n0, lds)
    if (NBM == 1 || left <= 16) MOE_FEW(1);
    else if (NBM == 2 || left <= 32) MOE_FEW(2);
    else if (NBM == 4 || left <= 64) MOE_FEW(4);
    else if (MODE == kFewCodes && left <= 96) MOE_FEW(6);
    else MOE_FEW(8);
#undef MOE_FEW
  }
}

template <int MODE, int KW, int NBM, bool WIDE = false>
hipError_t run_few_nb(const char* name, FewArgs a, int64_t active, hipStream_t s) {
  a.ctiles = (a.N + wg_cols<KW, WIDE>() - 1) / wg_cols<KW, WIDE>();
  // down's scales and its staging of every block count, and the waves' sums
  int lds = 0;
  for (int nb = 1; nb <= NBM; nb *= 2) {
    const int chunk = nb <= 2 ? 2048 : nb <= 4 ? 1024 : 512;
    const int stage = MODE == kFewDown ? 16 * nb * ((a.K < chunk ? a.K : chunk) + 16) : 0;
    const int sums = KW > 1 ? kFewWaves * wave_operands<MODE, WIDE>() * nb * 1024 : 0;
    lds = std::max(lds, std::max(stage, sums));
  }
  lds += kScaleBytes;
  auto k = few_rows_i8_kernel<MODE, KW, NBM, WIDE>;
  if (lds > 64 * 1024) {  // (the call is a good part of a small launch's host time)
    hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  {
    MOE_TRACE(name, s);
    MOE_LAUNCH(k, dim3((unsigned)(active * a.ctiles)), dim3(kFewThreads), lds, s, a);
  }
  return hipGetLastError();
}
template <int MODE, int KW>
hipError_t run_few_kw(const char* name, const FewArgs& a, int cap, bool wide, int64_t active, hipStream_t s) {
  if (cap <= 16) return run_few_nb<MODE, KW, 1>(name, a, active, s);
  if constexpr (MODE != kFewDown && KW < 4) {
    return run_few_nb<MODE, KW, 2>(name, a, active, s);  // cap <= 32
  } else {
    if (cap <= 32) return run_few_nb<MODE, KW, 2>(name, a, active, s);
    if constexpr (MODE == kFewCodes) {
      if (wide && cap <= 64) return run_few_nb<MODE, KW, 4, true>(name, a, active, s);
      if (wide) return run_few_nb<MODE, KW, 8, true>(name, a, active, s);
    }
    if (cap <= 64) return run_few_nb<MODE, KW, 4>(name, a, active, s);
    return run_few_nb<MODE, KW, 8>(name, a, active, s);
  }
}

// Rows of a pass: enough for nearly every group when rows spread by chance (their deviation is the square root
// of the mean), so that weights are read once; a fuller group takes more passes.
int pass_rows(int64_t usual, bool spread) {
  const double most = (double)usual + (spread ? 4.0 * std::sqrt((double)usual) : 0.0);
  int cap = 16;
  while (cap < kMaxRows && cap < most) cap *= 2;
  return cap;
}
constexpr int64_t kWant = 2 * 256;  // workgroups: one or two for every CU
// Column slices of 16 that a workgroup of down takes. With many columns 32 a wave, since every workgroup stages
// the rows first (33 tokens of 128 experts, H = 512, I = 256: the layer 25 -> 21 us; 4 tokens, H = 2048, I =
// 768 38 -> 34.5 us); then the widest slice that gives every CU a workgroup or two.
int down_slices(int64_t active, int64_t cols, int cap) {
  if (cap <= 32 && active * ((cols + 7) / 8) >= kWant) return 8;
  return active * ((cols + 3) / 4) >= kWant ? 4 : active * ((cols + 1) / 2) >= kWant ? 2 : 1;
}

// rows: a bound of the rows of all groups; usual: the rows that one group has on average
template <int MODE>
hipError_t run_few(const char* name, FewArgs a, int64_t rows, int64_t usual, hipStream_t s) {
  const int cap = pass_rows(usual, a.offsets != nullptr);
  a.listed = a.offsets && rows < a.groups;  // fewer rows than groups: list the groups that have some
  const int64_t active = a.listed ? rows : a.groups;
  // Plain products of more than 32 rows take 32 columns a wave where that leaves most CUs a workgroup (77 rows x
  // 2048 on 7168 columns 21 -> 14 us; on 2048 columns 12.5 -> 13.7 us, so not there); then the widest column
  // slice that still gives every CU a workgroup or two.
  const bool wide = MODE == kFewCodes && cap >= 64 && active * ((a.N + 2 * kCols - 1) / (2 * kCols)) >= 192;
  const int per = wide ? 2 : 1;
  const int64_t cols = (a.N + per * kCols - 1) / (per * kCols);
  if constexpr (MODE == kFewDown) {
    switch (down_slices(active, cols, cap)) {
      case 8: return cap <= 16 ? run_few_nb<MODE, 1, 1, true>(name, a, active, s) : run_few_nb<MODE, 1, 2, true>(name, a, active, s);
      case 4: return run_few_kw<MODE, 1>(name, a, cap, false, active, s);
      case 2: return run_few_kw<MODE, 2>(name, a, cap, false, active, s);
      default: return run_few_kw<MODE, 4>(name, a, cap, false, active, s);
    }
  } else {
    // (more than 32 rows on so many columns: a product goes to the GEMM, and gate/up comes here with a small H only)
    if (cap <= 32 && active * ((cols + 3) / 4) >= kWant) return run_few_kw<MODE, 1>(name, a, cap, wide, active, s);
    if (cap <= 32 && active * ((cols + 1) / 2) >= kWant) return run_few_kw<MODE, 2>(name, a, cap, wide, active, s);
    return run_few_kw<MODE, 4>(name, a, cap, wide, active, s);
  }
}

}  // namespace

// Bytes of rows that an expert layer's workgroups read here: gate/up every row of H codes for each 16 columns, down
// every row of I FP32 values for each workgroup.
int64_t few_rows_i8_traffic(int64_t groups, int64_t usual, int64_t H, int64_t I) {
  const int64_t cols = (H + kCols - 1) / kCols, per = down_slices(groups, cols, pass_rows(usual, true));
  return groups * usual * (I / kCols * H + (cols + per - 1) / per * I * 4);
}

// rows: a bound of the rows of chunks c0 .. c0 + nc - 1 together; usual: one expert's in one chunk on average
hipError_t launch_expert_fwd_i8_few(const void* xd, const float* xd_scale, const void* w1, const float* w1_scale,
                                    const void* w2, const float* w2_scale, const int32_t* offsets, void* h,
                                    void* yd, int H, int I, int El, int c0, int nc, int64_t P_c, int64_t P,
                                    int64_t rows, int64_t usual, hipStream_t s) {
  uint32_t* part = (uint32_t*)((char*)h + P * (int64_t)I * 4);
  FewArgs a{};
  a.x = (const int8_t*)xd; a.x_scale = xd_scale; a.part = part; a.w = (const int8_t*)w1; a.w_scale = w1_scale;
  a.out_h = (float*)h; a.offsets = offsets; a.P_c = P_c; a.K = H; a.N = I; a.El = El; a.c0 = c0; a.groups = El * nc;
  hipError_t e = run_few<kFewGateUp>("few_gateup_swiglu_i8", a, rows, usual, s);
  if (e != hipSuccess) return e;
  FewArgs b{};
  b.h = (const float*)h; b.part = part; b.w = (const int8_t*)w2; b.w_scale = w2_scale; b.y = (uint16_t*)yd;
  b.offsets = offsets; b.P_c = P_c; b.K = I; b.N = H; b.El = El; b.c0 = c0; b.groups = El * nc;
  return run_few<kFewDown>("few_down_i8", b, rows, usual, s);
}

hipError_t launch_expert_matmul_i8_few(int groups, int64_t rows, int N, int K, const void* x, const float* x_scale,
                                       const void* w, const float* w_scale, const int32_t* offsets, void* y,
                                       hipStream_t s) {
  FewArgs a{};
  a.x = (const int8_t*)x; a.x_scale = x_scale; a.w = (const int8_t*)w; a.w_scale = w_scale; a.y = (uint16_t*)y;
  a.offsets = offsets; a.P_c = rows; a.K = K; a.N = N; a.El = groups; a.groups = groups;
  return run_few<kFewCodes>("few_matmul_i8", a, rows, (rows + groups - 1) / groups, s);
}

}  // namespace moe
