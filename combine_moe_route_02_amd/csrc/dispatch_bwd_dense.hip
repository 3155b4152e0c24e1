// Dispatch backward with a dense router gradient (MOE_FLAG_ROUTER_LOSS): an auxiliary loss reaches the
// logits of every expert, so
//   dx[t] = RNE( sum over local slots j of dxd[row_of[t][j]] + sum over all e of dlogits[t][e] W_r[e] ).
// The second sum is a [T, E] x [E, H] product whose epilogue gathers the expert rows, so dx is written
// once and no [T, H] term goes through memory. dlogits is FP32: it is split into a BF16 high and low
// part (the remainder is under 2^-17 of the value, far under the BF16 rounding of dx; W_r is BF16
// itself) and both run on BF16 MFMA into the same FP32 sums.
//
// A workgroup (4 waves) keeps its column slice of W_r in registers as MFMA fragments for every expert
// and walks 32-token tiles: the tile's dlogits are split into LDS once for the four waves, each wave
// multiplies its columns, the FP32 sums go through LDS into rows of 16-byte vectors, and there the
// slots' dxd rows are added as they are loaded. Each XCD owns a range of tokens, so that the tile's
// dlogits, which every slice reads, come from its L2. A slot's dxd rows and the next tile's dlogits are loaded a
// tile ahead. dx is stored past the L2, which keeps the rows and dlogits (44 -> 39 us; loads of
// the rows marked the same way 48 us). 16384 tokens x 2048, 128 experts of which 16 are local: 37 us for 144 MB (3.9 TB/s;
// 29 us at the rate of a copy), bound by the rows' gather behind two barriers per tile; 1000 tokens x 256: 5.5 us, one tile per
// workgroup, latency. Slices of 128 columns (three workgroups per CU) 57 us, two rows ahead 48 us.
#include <type_traits>

#include "gg_engine.h"

namespace moe {
namespace {

using gg::frag_ks;
using gg::ks_off;

constexpr int kDT = 32;        // tokens per tile
constexpr int kDThreads = 256;
constexpr int kStageK = 64;    // W_r rows staged at once
constexpr int kAhead = 3;      // dxd rows of a token loaded a tile ahead

// KS: K steps of 16 experts (E <= 16 KS); CW: columns per wave
template <int KS, int CW>
struct DenseLds {
  static constexpr int kSlice = 4 * CW;
  static constexpr int kPitchA = KS * 32 + 16;        // bytes per token of one part
  static constexpr int kPartA = kDT * kPitchA;
  static constexpr int kPitchC = (kSlice + 4) * 4;    // bytes per token of the FP32 sums
  static constexpr int kC = 2 * kPartA;
  static constexpr int kSums = kDT * kPitchC;
  static constexpr int kW = (KS * 16 < kStageK ? KS * 16 : kStageK) * kSlice * 2;  // W_r staging, before the first tile
  static constexpr int kRows = kC + (kSums > kW ? kSums : kW);
  static constexpr int kBytes = kRows + 3 * kDT * 8 * 4;  // slot rows of three tiles
};

// One vector of 8 columns of a dispatch row: BF16 values, or (Q) e4m3 codes with their block's scale. Loads
// and adds carry no branch (a row that is absent loads row 0 and adds zeros): the compiler counts
// loads in flight only in straight code, and behind branches waits for all of them.
template <bool Q> struct RowVec;
template <> struct RowVec<false> {
  u32x4 v;
  MOE_DEV void load(const void* dxd, const float*, int64_t r, int64_t nvec, int vec, int) {
    v = ((const u32x4*)dxd)[r * nvec + vec];
  }
  MOE_DEV void add(float (&f)[8], bool on) const {
    const uint32_t m = on ? 0xffffffffu : 0u, w[4] = {v.x & m, v.y & m, v.z & m, v.w & m};
#pragma unroll
    for (int i = 0; i < 4; ++i) { f[2 * i] += bf2f(w[i] & 0xffff); f[2 * i + 1] += bf2f(w[i] >> 16); }
  }
};
template <> struct RowVec<true> {
  uint2 v;
  float s;
  MOE_DEV void load(const void* dxd, const float* dxs, int64_t r, int64_t nvec, int vec, int nblk) {
    v = ((const uint2*)dxd)[r * nvec + vec];
    s = dxs[r * nblk + (vec >> 5)];
  }
  MOE_DEV void add(float (&f)[8], bool on) const {
    float g[8];
    const uint32_t m = on ? 0xffffffffu : 0u;
    deq8(make_uint2(v.x & m, v.y & m), on ? s : 0.f, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += g[i];
  }
};

struct DenseArgs {
  const void* dxd;        // [P, H] BF16 rows, or e4m3 codes (Q)
  const float* dxs;       // Q: [P, ceil(H / 256)]
  const int32_t* row_of;  // [T, K]
  const float* dlogits;   // [T, E]
  const uint16_t* w_r;    // [E, H]
  uint16_t* dx;           // [T, H]
  int64_t t0, t1;
  int K, E, H, nsl, lanes;  // column slices; workgroups per XCD and slice
};

template <int KS, int CW, bool Q>
__global__ __launch_bounds__(kDThreads, KS <= 8 ? 2 : 1) void dispatch_bwd_dense_kernel(DenseArgs a) {
  using L = DenseLds<KS, CW>;
  constexpr int TN = CW / 32, SL = L::kSlice;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  char* const sc = lds + L::kC;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t tiles = (a.t1 - a.t0 + kDT - 1) / kDT, px = (tiles + 7) / 8;
  const int xcd = blockIdx.x % 8, j = blockIdx.x / 8;
  const int n0 = (j % a.nsl) * SL, first = j / a.nsl;
  if (xcd * px + first >= tiles || first >= px) return;

  const int64_t nvec = a.H / 8;
  const int nblk = (a.H + 255) / 256;
  const int evec = a.E / 4;
  constexpr int ND = kDT * KS * 4 / kDThreads;  // 16-byte vectors of the tile's dlogits per thread
  constexpr int VPR = SL / 8;                   // vectors of 8 columns per token
  constexpr int NI = kDT * VPR / kDThreads;     // of them per thread: tokens tid / VPR + it * (256 / VPR)
  const int c = tid % VPR, rt = tid / VPR, n = n0 + 8 * c;
  const bool in_cols = n < a.H;
  const int vec = min(n, a.H - 8) / 8;
  const void* const dxd = a.dxd ? a.dxd : a.w_r;  // no local expert: any readable row
  float4 dl[ND];
  int slots[8];
  // dlogits of a tile (one contiguous block; columns past E and tokens past the chunk are zeros): issued one
  // tile ahead
  auto fetch = [&](int64_t tile) {
    const int64_t r0 = a.t0 + tile * kDT;
    const int nt = (int)(a.t1 - r0 < kDT ? a.t1 - r0 : kDT);
#pragma unroll
    for (int u = 0; u < ND; ++u) {  // unconditional (so that later waits can count them); zeroed where it is used
      const int i = tid + u * kDThreads, r = min(i / (KS * 4), nt - 1), e4 = min(i % (KS * 4), evec - 1);
      dl[u] = *(const float4*)(a.dlogits + (r0 + r) * a.E + 4 * e4);
    }
  };
  // slots of token tid (tid < kDT) of the XCD's tile l: issued two tiles ahead, put into LDS one tile ahead,
  // the token's local rows first, in slot order (none past the end)
  auto token = [&](int64_t l) { return a.t0 + (xcd * px + l) * kDT + min(tid, kDT - 1); };
  auto inside = [&](int64_t l) { return l < px && token(l) < a.t1; };
  auto fetch_slots = [&](int64_t l) {
    if (wave > 0) return;
    const int32_t* p = a.row_of + (inside(l) ? token(l) : a.t0) * a.K;
#pragma unroll
    for (int k = 0; k < 8; ++k) slots[k] = p[min(k, a.K - 1)];
  };
  auto put_slots = [&](int buf, int64_t l) {
    if (wave > 0 || tid >= kDT) return;
    int* const srow = (int*)(lds + L::kRows) + buf * (kDT * 8) + tid * 8;
    const bool in = inside(l);
    int m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      srow[m] = slots[k];  // kept if it is a local slot, else overwritten
      m += in && k < a.K && slots[k] >= 0 ? 1 : 0;
    }
    for (; m < 8; ++m) srow[m] = -1;
  };
  fetch_slots(first);
  fetch(xcd * px + first);

  // the slice of W_r as fragments: rows of W_r through LDS, transposed by the fragment reads; two
  // stages' rows are loaded together
  bf16x8_t w[KS][TN];
  {
    constexpr int SK = KS * 16 < kStageK ? KS * 16 : kStageK;  // rows per stage
    constexpr int NS = KS * 16 / SK, SB = NS < 2 ? NS : 2;     // stages, of them loaded at once
    constexpr int CPR = SL / 8, NV = SK * CPR / kDThreads;     // 16-byte vectors per row, per thread and stage
#pragma unroll
    for (int s0 = 0; s0 < NS; s0 += SB) {
      u32x4 x[SB][NV];
#pragma unroll
      for (int s = 0; s < SB; ++s)
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          const int i = tid + u * kDThreads, e = (s0 + s) * SK + i / CPR, col = n0 + 8 * (i % CPR);
          x[s][u] = u32x4{0u, 0u, 0u, 0u};
          if (e < a.E && col < a.H) x[s][u] = *(const u32x4*)(a.w_r + (int64_t)e * a.H + col);
        }
#pragma unroll
      for (int s = 0; s < SB; ++s) {
        gg::lds_barrier();  // the stage before this one has been read
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          const int i = tid + u * kDThreads;
          *(u32x4*)(sc + ks_off<SL>(i / CPR, i % CPR)) = x[s][u];
        }
        gg::lds_barrier();
#pragma unroll
        for (int kk = 0; kk < SK / 16; ++kk)
#pragma unroll
          for (int tn = 0; tn < TN; ++tn) w[(s0 + s) * (SK / 16) + kk][tn] = frag_ks<SL>(sc, wave * CW + 32 * tn, kk, lane);
      }
    }
  }
  // The tokens' first kAhead dxd rows are loaded a tile ahead.
  RowVec<Q> v[kAhead][NI];
  int row[kAhead][NI];
  auto fetch_rows = [&](int buf) {
    const int* const srow = (const int*)(lds + L::kRows) + buf * (kDT * 8);
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int u = 0; u < NI; ++u) {
        row[s][u] = srow[(rt + u * (kDThreads / VPR)) * 8 + s];
        v[s][u].load(dxd, a.dxs, max(row[s][u], 0), nvec, vec, nblk);
      }
  };
  put_slots(0, first);
  fetch_slots(first + a.lanes);
  gg::lds_barrier();
  fetch_rows(0);
  // Two barriers per tile. A wave may start the next tile while others still add rows of this one or look
  // up the next one's, so the slot rows go round three buffers; the parts and the sums are separate areas.
  int buf = 0;
  for (int64_t l = first; l < px; l += a.lanes) {
    const int64_t tile = xcd * px + l;
    if (tile >= tiles) break;
    const int* const srow = (const int*)(lds + L::kRows) + buf * (kDT * 8);
    buf = buf == 2 ? 0 : buf + 1;
    const int64_t r0 = a.t0 + tile * kDT;
    const int nt = (int)(a.t1 - r0 < kDT ? a.t1 - r0 : kDT);
#pragma unroll
    for (int u = 0; u < ND; ++u) {
      const int i = tid + u * kDThreads, r = i / (KS * 4), e4 = i % (KS * 4);
      if (r >= nt || e4 >= evec) dl[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      const uint2 h = gg::pack4(dl[u].x, dl[u].y, dl[u].z, dl[u].w);
      float hf[4];
      gg::unpack4(h, hf);
      *(uint2*)(lds + r * L::kPitchA + 8 * e4) = h;
      *(uint2*)(lds + L::kPartA + r * L::kPitchA + 8 * e4) =
          gg::pack4(dl[u].x - hf[0], dl[u].y - hf[1], dl[u].z - hf[2], dl[u].w - hf[3]);
    }
    put_slots(buf, l + a.lanes);  // the next tile's
    gg::lds_barrier();  // (loads stay in flight)
    fetch(tile + a.lanes < tiles ? tile + a.lanes : tile);  // (unused behind the last tile)
    fetch_slots(l + 2 * a.lanes);

    f32x16_t acc[TN];
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[tn][q] = 0.f;
    const char* fa = lds + (lane & 31) * L::kPitchA + 16 * (lane >> 5);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const bf16x8_t hi = *(const bf16x8_t*)(fa + 32 * kk), lo = *(const bf16x8_t*)(fa + L::kPartA + 32 * kk);
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        acc[tn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[kk][tn], hi, acc[tn], 0, 0, 0);
        acc[tn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[kk][tn], lo, acc[tn], 0, 0, 0);
      }
    }
    // lane: token lane & 31, four consecutive columns per accumulator group
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(float4*)(sc + (lane & 31) * L::kPitchC + 4 * (wave * CW + 32 * tn + gg::out_col(g, lane))) =
            make_float4(acc[tn][4 * g], acc[tn][4 * g + 1], acc[tn][4 * g + 2], acc[tn][4 * g + 3]);
    gg::lds_barrier();  // the loads above stay in flight
    __builtin_amdgcn_sched_barrier(0);  // nothing that waits for the rows moves in front of the products

    float f[NI][8];
#pragma unroll
    for (int u = 0; u < NI; ++u) {
      const int r = rt + u * (kDThreads / VPR);
      const float4 x = *(const float4*)(sc + r * L::kPitchC + 32 * c), y = *(const float4*)(sc + r * L::kPitchC + 32 * c + 16);
      f[u][0] = x.x; f[u][1] = x.y; f[u][2] = x.z; f[u][3] = x.w;
      f[u][4] = y.x; f[u][5] = y.y; f[u][6] = y.z; f[u][7] = y.w;
    }
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int u = 0; u < NI; ++u)
        v[s][u].add(f[u], row[s][u] >= 0);
    // tokens with more local slots: the next slot of every token in flight together
    for (int s = kAhead; s < a.K; ++s) {
      bool any = false;
#pragma unroll
      for (int u = 0; u < NI; ++u) {
        row[0][u] = srow[(rt + u * (kDThreads / VPR)) * 8 + s];
        any |= row[0][u] >= 0;
      }
      if (__ballot(any) == 0) break;
#pragma unroll
      for (int u = 0; u < NI; ++u) v[0][u].load(dxd, a.dxs, max(row[0][u], 0), nvec, vec, nblk);
#pragma unroll
      for (int u = 0; u < NI; ++u) v[0][u].add(f[u], row[0][u] >= 0);
    }
#pragma unroll
    for (int u = 0; u < NI; ++u) {
      const int r = rt + u * (kDThreads / VPR);
      if (r < nt && in_cols)
        __builtin_nontemporal_store(i32x4_t{(int)pack_bf2(f[u][0], f[u][1]), (int)pack_bf2(f[u][2], f[u][3]),
                                            (int)pack_bf2(f[u][4], f[u][5]), (int)pack_bf2(f[u][6], f[u][7])},
                                    (i32x4_t*)(a.dx + (r0 + r) * a.H + n));
    }
    fetch_rows(buf);
  }
}

// FP32 payloads: FP32 MFMA (32 x 32 x 2), so that the sums keep FP32 products. A workgroup takes 32 tokens and 128
// columns, a wave 32 of them; dlogits and W_r pass through LDS in chunks of 64 experts, the next chunk's loads in
// registers meanwhile, and a token's first rows of dxd are on their way from the start. Experts e and e + half of a
// chunk make one step, so that the dlogits reads of both lane halves fall on different banks. Three workgroups per CU
// (LDS; 168 registers) cover one another's loads: 3731 tokens x 1088 with 116 experts 23 us, 27 us with two. 16000
// tokens x 2048: 241 us with 32 experts, all local, 8 per token (the rate of a copy); 165 us with 160 experts of which
// 20 are local, 64 TFLOP/s (57 us of bytes and 69 us of FP32 products; 64 tokens a workgroup 158 us, but 3731 tokens
// 28 us).
constexpr int kFCols = 128, kFE = 64;
struct alignas(16) F32Lds {
  union {
    float w[kFE][kFCols];
    float sums[kDT][kFCols + 4];
  };
  float dl[kDT][kFE + 1];
  int32_t row[kDT][8];
};

__global__ __launch_bounds__(kDThreads, 3) void dispatch_bwd_dense_f32_kernel(
    const float* __restrict__ dxd, const int32_t* __restrict__ row_of, const float* __restrict__ dlogits,
    const float* __restrict__ w_r, float* __restrict__ dx, int64_t t0, int64_t t1, int K, int E, int H, int nct) {
  constexpr int NO = 4, kAheadF = 2;  // output vectors of a thread; rows of a token loaded from the start
  __shared__ F32Lds sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t tiles = (t1 - t0 + kDT - 1) / kDT, px = (tiles + 7) / 8;
  const int64_t tile = blockIdx.x % 8 * px + blockIdx.x / 8 / nct;  // an XCD's tokens are one range
  if (tile >= tiles) return;
  const int64_t r0 = t0 + tile * kDT;
  const int nt = (int)(t1 - r0 < kDT ? t1 - r0 : kDT), n0 = blockIdx.x / 8 % nct * kFCols;

  // chunk loads: 8 vectors of W_r (rows tid / 32 + 8 u), 8 values of dlogits (tokens tid / 64 + 4 u); loads carry no
  // branch (the compiler would wait behind each), and experts past the last one are zeroed as they go to LDS
  float4 wv[8];
  float dv[8];
  const int wc = n0 + 4 * (tid % 32);
  auto fetch = [&](int e0) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int e = e0 + tid / 32 + 8 * u, d = e0 + lane, t = wave + 4 * u;
      wv[u] = *(const float4*)(w_r + (int64_t)min(e, E - 1) * H + min(wc, H - 4));
      dv[u] = dlogits[(r0 + min(t, nt - 1)) * E + min(d, E - 1)];
    }
  };
  fetch(0);
  // a token's local rows first, in slot order
  if (tid < kDT) {
    int32_t slots[8];
    const int32_t* p = row_of + (r0 + min(tid, nt - 1)) * K;
#pragma unroll
    for (int k = 0; k < 8; ++k) slots[k] = p[min(k, K - 1)];
    int m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      sh.row[tid][m] = slots[k];  // kept if it is a local slot, else overwritten
      m += k < K && slots[k] >= 0 ? 1 : 0;
    }
    for (; m < 8; ++m) sh.row[tid][m] = -1;
  }
  gg::lds_barrier();
  // out: thread holds 4 columns of tokens tid / 32 + 8 u
  const int oc = 4 * (tid % 32), ot = tid / 32;
  const bool in_cols = n0 + oc < H;
  const float* const rows = dxd ? dxd : w_r;  // no local expert: any readable row
  float4 v[kAheadF][NO];
  bool on[kAheadF][NO];
  auto load_rows = [&](float4 (&d)[NO], bool (&on)[NO], int s) {
#pragma unroll
    for (int u = 0; u < NO; ++u) {
      const int r = sh.row[ot + 8 * u][s];
      on[u] = r >= 0;
      d[u] = *(const float4*)(rows + (int64_t)max(r, 0) * H + min(n0 + oc, H - 4));
    }
  };
#pragma unroll
  for (int s = 0; s < kAheadF; ++s) load_rows(v[s], on[s], s);

  f32x16_t acc;
#pragma unroll
  for (int q = 0; q < 16; ++q) acc[q] = 0.f;
  for (int e0 = 0; e0 < E; e0 += kFE) {
    if (e0 > 0) gg::lds_barrier();  // the chunk before this one has been read
#pragma unroll
    for (int u = 0; u < 8; ++u)
      *(float4*)&sh.w[tid / 32 + 8 * u][4 * (tid % 32)] = e0 + tid / 32 + 8 * u < E ? wv[u] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < 8; ++u) sh.dl[wave + 4 * u][lane] = e0 + lane < E ? dv[u] : 0.f;
    gg::lds_barrier();
    if (e0 + kFE < E) fetch(e0 + kFE);
    const int half = (min(kFE, E - e0) + 1) / 2, eh = (lane >> 5) * half;
    const float* pw = &sh.w[eh][32 * wave + (lane & 31)];
    const float* pd = &sh.dl[lane & 31][eh];
    auto steps = [&](int i, auto n) {
      constexpr int N = decltype(n)::value;
      float w[N], d[N];
#pragma unroll
      for (int j = 0; j < N; ++j) { w[j] = pw[(i + j) * kFCols]; d[j] = pd[i + j]; }
#pragma unroll
      for (int j = 0; j < N; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(w[j], d[j], acc, 0, 0, 0);
    };
    int i = 0;
    for (; i + 4 <= half; i += 4) steps(i, std::integral_constant<int, 4>());
    for (; i < half; ++i) steps(i, std::integral_constant<int, 1>());
  }
  gg::lds_barrier();
  // lane: token lane & 31, four consecutive columns per accumulator group
#pragma unroll
  for (int g = 0; g < 4; ++g)
    *(float4*)&sh.sums[lane & 31][32 * wave + gg::out_col(g, lane)] =
        make_float4(acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]);
  gg::lds_barrier();
  float4 f[NO];
#pragma unroll
  for (int u = 0; u < NO; ++u) f[u] = *(const float4*)&sh.sums[ot + 8 * u][oc];
  auto add = [&](const float4 (&d)[NO], const bool (&on)[NO]) {
#pragma unroll
    for (int u = 0; u < NO; ++u) {
      f[u].x += on[u] ? d[u].x : 0.f; f[u].y += on[u] ? d[u].y : 0.f;
      f[u].z += on[u] ? d[u].z : 0.f; f[u].w += on[u] ? d[u].w : 0.f;
    }
  };
#pragma unroll
  for (int s = 0; s < kAheadF; ++s) add(v[s], on[s]);
  for (int s = kAheadF; s < K; ++s) {
    bool any = false;
#pragma unroll
    for (int u = 0; u < NO; ++u) any |= sh.row[ot + 8 * u][s] >= 0;
    if (__ballot(any) == 0) break;
    load_rows(v[0], on[0], s);
    add(v[0], on[0]);
  }
#pragma unroll
  for (int u = 0; u < NO; ++u) {
    const int t = ot + 8 * u;
    if (t < nt && in_cols) __builtin_nontemporal_store(f32x4_t{f[u].x, f[u].y, f[u].z, f[u].w}, (f32x4_t*)(dx + (r0 + t) * H + n0 + oc));
  }
}

template <int KS, int CW, bool Q>
hipError_t run_dense(DenseArgs a, hipStream_t s) {
  using L = DenseLds<KS, CW>;
  auto k = dispatch_bwd_dense_kernel<KS, CW, Q>;
  hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != hipSuccess) return e;
  a.nsl = (a.H + L::kSlice - 1) / L::kSlice;
  // two workgroups per CU, and the tiles of an XCD spread evenly over its workgroups of a slice
  const int64_t px = ((a.t1 - a.t0 + kDT - 1) / kDT + 7) / 8;
  int64_t lanes = (int64_t)gg::cu_count() / 8 * 2 / a.nsl;
  if (lanes < 1) lanes = 1;
  if (lanes > px) lanes = px;
  const int64_t per = (px + lanes - 1) / lanes;
  a.lanes = (int)((px + per - 1) / per);
  {
    MOE_TRACE("dispatch_bwd_dense", s);
    MOE_LAUNCH(k, dim3((unsigned)(8 * a.nsl * a.lanes)), dim3(kDThreads), L::kBytes, s, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch_bwd_dense(bool bf16, const void* dxd, const float* dxd_scales, const int32_t* row_of,
                                     const float* dlogits, const void* w_r, void* dx, int64_t t0, int64_t t1, int K,
                                     int E, int H, hipStream_t s) {
  if (t1 <= t0) return hipSuccess;
  if (!bf16) {
    MOE_TRACE("dispatch_bwd_dense_f32", s);
    const int nct = (H + kFCols - 1) / kFCols;
    const int64_t px = ((t1 - t0 + kDT - 1) / kDT + 7) / 8;
    MOE_LAUNCH(dispatch_bwd_dense_f32_kernel, dim3((unsigned)(8 * px * nct)), dim3(kDThreads), 0, s, (const float*)dxd,
               row_of, dlogits, (const float*)w_r, (float*)dx, t0, t1, K, E, H, nct);
    return hipGetLastError();
  }
  DenseArgs a{dxd, dxd_scales, row_of, dlogits, (const uint16_t*)w_r, (uint16_t*)dx, t0, t1, K, E, H, 0, 0};
  // fragments of a wave: 64 columns of up to 256 experts, 32 of up to 1024 (at most 256 registers)
#define MOE_DENSE(KS_, CW_) return dxd_scales ? run_dense<KS_, CW_, true>(a, s) : run_dense<KS_, CW_, false>(a, s)
  if (E <= 32) MOE_DENSE(2, 64);
  if (E <= 64) MOE_DENSE(4, 64);
  if (E <= 128) MOE_DENSE(8, 64);
  if (E <= 256) MOE_DENSE(16, 64);
  if (E <= 512) MOE_DENSE(32, 32);
  MOE_DENSE(64, 32);
#undef MOE_DENSE
}

}  // namespace moe
