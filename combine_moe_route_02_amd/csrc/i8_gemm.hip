// Grouped GEMMs of the 8-bit integer experts: v_mfma_i32_32x32x32_i8 on tiles of 256 x 256 (8 waves of 128 x 64,
// operands by direct-to-LDS loads into two slots of 128-byte rows) or, where those are too few for the CUs, of
// 128 x 128 (4 waves of 64 x 64, four slots) or 64 x 64 (4 waves of 32 x 32, eight slots).
//
// Integer products take half the time of BF16 ones, so what surrounds a tile's K loop (its first loads, sums
// through LDS into rows with a barrier on each side, stores) weighs double. Here the list of tiles is one
// stream instead:
//   * during a tile's last pairs of stages its workgroup already loads the next tile's first ones and its scales,
//     into the slots that further pairs would have had;
//   * the sums go from registers to HBM without LDS: swapping lane halves gives every lane 8 columns of a
//     row (16 bytes), so neither ring slot nor barrier is needed. Each wave issues exactly kStores buffer
//     stores per tile, rows and columns outside it dropped by the descriptor's extent, and the
//     next tile waits for its loads with those stores still in flight.
// Measured at 8192 x 4096 x 7168: 195 us (2.47 POPS; MFMA busy 65% of the cycles, clock 1.8 GHz under
// this load, LDS bank conflicts 0; 210 us on a slower card) against 220 us tile by tile on a card of 198; four slots of single
// stages, loaded three ahead, 222 us. The expert products of the 16K-token share take two rounds of 33 us (gate/up, 66) and
// two and a part of 22 us (down, 51): 128-row tiles lose more in the K loop than they gain in the last round (gate/up
// 90 us, down 59 us).
// Small tiles: 0.5 us a pair of stages. One wave a SIMD does its fragment reads, its products and its waits one after the
// other: on a CU that has a tile MFMA is busy 28% and LDS 15% of the cycles, and loads of nothing take the same time. They
// stream weights at HBM's rate (128 groups of 24 rows x 2048 on 1536 columns 82 us, 4.9 TB/s). Eight waves of 32 x 64
// take the same time. Tiny tiles: 0.3 us a pair, so four of them on four CUs beat a small one (256 rows x 7168 on 4096
// columns 28 -> 21 us).
// Tiles of 256 x 192 gain with even groups (gate/up of 16 x 1024 rows 60 -> 55 us) and lose with uneven ones,
// whose small last tiles then make a third round (65 -> 83 us).
// The sums are exact in int32 and rounded once to FP32; scales multiply in FP32 and BF16 rounds once.
#include <type_traits>

#include "gg_engine.h"
#include "i8.h"

namespace moe {
namespace gg {
namespace {

// Tiles of kTile x kTile, waves kWM x kWN, each with kMN x kNN blocks of 32 x 32
enum { kLarge = 256, kSmall = 128, kTiny = 64 };
template <int TILE> struct I8Shape {
  static constexpr int kTile = TILE, kWM = 2, kWN = TILE == kLarge ? 4 : 2;
  static constexpr int kThreads = 64 * kWM * kWN;
  static constexpr int kMN = kTile / kWM / 32, kNN = kTile / kWN / 32;
  static constexpr int kSlotA = kTile * 2 * kRowB, kSlot = 2 * kSlotA;  // pair slot: rows of A, then of B
  static constexpr int kSlots = 512 / kTile, kRing = kSlots * kSlot;    // 128 KB
  static constexpr int kStores = 2 * kMN * kNN;                         // buffer stores of a wave per tile
  static_assert(kThreads >= 2 * kTile, "one scale per thread");
};
constexpr int kOutside = 0x7ffffff0;  // past every output descriptor's extent (at most 2^30 bytes)
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;

struct I8Args {
  const int8_t* A;         // [P, K]
  const float* scale_a;    // [P]
  const int8_t* B;         // per expert [N, K], gate/up [2 N, K]
  const float* scale_b;    // per expert [N], [2 N]
  void* C;                 // gate/up: h [P, N] FP32; product [P, N] BF16; down: rows of yd (i8.h)
  int K, N;
  const int32_t* offsets;  // null: one group of P_c rows
  int El, c0, nc;
  int64_t P_c;
};

struct Groups {
  int pre[kMaxGroups + 1], preb[kMaxGroups + 1];  // tiles before group g: large, small
  int o0[kMaxGroups], len[kMaxGroups];
};

struct I8Tile {
  const char* a;  // first byte of its rows, and their extent
  const char* b;
  int64_t abytes, bbytes, r0;
  int mvalid, n0, e;
};

// Running sums of v[1 .. G] in place, by one wave.
MOE_DEV void scan(int* v, int G, int lane) {
  int before = 0;
  if (lane == 0) v[0] = 0;
  for (int g0 = 0; g0 < G; g0 += 64) {
    int x = g0 + lane < G ? v[g0 + lane + 1] : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(x, o, 64);
      if (lane >= o) x += y;
    }
    if (g0 + lane < G) v[g0 + lane + 1] = before + x;
    before += __builtin_amdgcn_readlane(x, 63);
  }
}

// The same of one value per lane, in registers (a chain of DPP steps).
MOE_DEV int scan64(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8: sums inside 16 lanes
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // lane 15 to lanes 16 .. 31, 47 to 48 .. 63
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // lane 31 to lanes 32 .. 63
  return x;
}

// Group of a tile: the groups whose tiles end at or before it.
MOE_DEV int group_of(const int* pre, int G, int tile, int lane) {
  int g = 0;
  for (int g0 = 0; g0 < G; g0 += 64) g += __popcll(__ballot(g0 + lane < G && pre[g0 + lane + 1] <= tile));
  return __builtin_amdgcn_readfirstlane(g);
}

// A lane's scales of a tile from LDS: its rows (of four blocks, or one), and four groups of four columns of
// each column block. Written in assembly because the compiler would first wait for every direct-to-LDS
// load in flight, those of the next tile's first stages here, which fill another part of LDS.
MOE_DEV void read_scales(uint32_t rows, uint32_t cols, float (&r)[4], f32x4_t (&c)[8]) {
  asm volatile(
      "ds_read_b32 %0, %12\n\tds_read_b32 %1, %12 offset:128\n\t"
      "ds_read_b32 %2, %12 offset:256\n\tds_read_b32 %3, %12 offset:384\n\t"
      "ds_read_b128 %4, %13\n\tds_read_b128 %5, %13 offset:32\n\t"
      "ds_read_b128 %6, %13 offset:64\n\tds_read_b128 %7, %13 offset:96\n\t"
      "ds_read_b128 %8, %13 offset:128\n\tds_read_b128 %9, %13 offset:160\n\t"
      "ds_read_b128 %10, %13 offset:192\n\tds_read_b128 %11, %13 offset:224\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(c[0]), "=&v"(c[1]), "=&v"(c[2]), "=&v"(c[3]),
        "=&v"(c[4]), "=&v"(c[5]), "=&v"(c[6]), "=&v"(c[7])
      : "v"(rows), "v"(cols)
      : "memory");
}
MOE_DEV void read_scales(uint32_t rows, uint32_t cols, float (&r)[4], f32x4_t (&c)[4]) {
  asm volatile(
      "ds_read_b32 %0, %5\n\tds_read_b128 %1, %6\n\tds_read_b128 %2, %6 offset:32\n\t"
      "ds_read_b128 %3, %6 offset:64\n\tds_read_b128 %4, %6 offset:96\n\ts_waitcnt lgkmcnt(0)"
      : "=&v"(r[0]), "=&v"(c[0]), "=&v"(c[1]), "=&v"(c[2]), "=&v"(c[3])
      : "v"(rows), "v"(cols)
      : "memory");
}

enum I8Out { kProduct, kGateUp8, kDown8 };  // BF16 rows; h in FP32; rows of yd (i8.h)
template <int OUT, int TILE>
__global__ __launch_bounds__(I8Shape<TILE>::kThreads) void i8_gemm_kernel(I8Args a) {
  using S = I8Shape<TILE>;
  constexpr bool GU = OUT == kGateUp8;
  constexpr int kTile = S::kTile, kWN = S::kWN, kThreads = S::kThreads, kMN = S::kMN, kNN = S::kNN, kSlots = S::kSlots;
  constexpr int OUTN = GU ? kTile / 2 : kTile;  // output columns of a tile
  __shared__ Groups sh;
  __shared__ float scales[kSlots][2 * kTile];  // rows, then columns in the order of the tile's rows of B
  extern __shared__ __attribute__((aligned(1024))) char ring[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / kWN, wn = wave % kWN;
  const int G = a.nc * a.El, ntiles = (a.N + OUTN - 1) / OUTN;
  // "large" row tiles (full, or a last one of more than half the rows) come before the "small" last ones,
  // which fill a last round where one is needed
  auto rows_of = [&](int g, int& o0, int& len, int& large, int& small) {
    const int c = a.c0 + g / a.El, e = g % a.El;
    o0 = 0;
    int o1 = (int)a.P_c;
    if (a.offsets) {  // nothing outside the rows, whatever the table holds
      const int32_t* off = a.offsets + (int64_t)c * (a.El + 1);
      o0 = max(0, min(off[e], (int)a.P_c));
      o1 = max(o0, min(off[e + 1], (int)a.P_c));
    }
    len = o1 - o0;
    const int rem = len % kTile;
    large = (len / kTile + (rem > kTile / 2 ? 1 : 0)) * ntiles;
    small = (rem > 0 && rem <= kTile / 2 ? 1 : 0) * ntiles;
  };
  // Up to 64 groups stay in registers, one per lane of every wave: the first tile's loads then wait for
  // neither LDS nor a barrier.
  const bool in_lanes = G <= 64;
  int l_o0 = 0, l_len = 0, l_pre = 0, l_preb = 0, total_l, total_s;
  if (in_lanes) {
    if (lane < G) rows_of(lane, l_o0, l_len, l_pre, l_preb);
    l_pre = scan64(l_pre);
    l_preb = scan64(l_preb);
    total_l = __builtin_amdgcn_readlane(l_pre, 63);
    total_s = __builtin_amdgcn_readlane(l_preb, 63);
  } else {
    for (int g = tid; g < G; g += kThreads) rows_of(g, sh.o0[g], sh.len[g], sh.pre[g + 1], sh.preb[g + 1]);
    __syncthreads();
    if (wave == 0) scan(sh.pre, G, lane);
    if (wave == 1) scan(sh.preb, G, lane);
    __syncthreads();
    total_l = __builtin_amdgcn_readfirstlane(sh.pre[G]);
    total_s = __builtin_amdgcn_readfirstlane(sh.preb[G]);
  }
  // each XCD (block % 8) owns a contiguous range of the large and one of the small tiles
  const int pxl = (total_l + 7) / 8, pxs = (total_s + 7) / 8;
  const int xcd = blockIdx.x % 8, per_xcd = gridDim.x / 8;

  auto find = [&](I8Tile& t, int& slot) -> bool {  // the tile of `slot`, or of the next slot that has one
    for (; slot < pxl + pxs; slot += per_xcd) {
      const bool large = slot < pxl;
      const int tile = large ? xcd * pxl + slot : xcd * pxs + (slot - pxl);
      if (tile >= (large ? total_l : total_s)) continue;
      int g, before, len, o0;
      if (in_lanes) {
        const int pre = large ? l_pre : l_preb;
        g = __popcll(__ballot(pre <= tile));  // (lanes past the groups hold the total)
        before = g > 0 ? __builtin_amdgcn_readlane(pre, g - 1) : 0;
        len = __builtin_amdgcn_readlane(l_len, g);
        o0 = __builtin_amdgcn_readlane(l_o0, g);
      } else {
        const int* pre = large ? sh.pre : sh.preb;
        g = group_of(pre, G, tile, lane);
        before = __builtin_amdgcn_readfirstlane(pre[g]);
        len = __builtin_amdgcn_readfirstlane(sh.len[g]);
        o0 = __builtin_amdgcn_readfirstlane(sh.o0[g]);
      }
      const int at = tile - before;
      const int mt = large ? at / ntiles : len / kTile;
      t.e = g % a.El;
      t.n0 = (at % ntiles) * OUTN;
      t.r0 = (int64_t)(a.c0 + g / a.El) * a.P_c + o0 + (int64_t)mt * kTile;
      t.mvalid = min(kTile, len - mt * kTile);
      const int64_t wrows = GU ? 2 * (int64_t)a.N : a.N;
      t.a = (const char*)a.A + t.r0 * a.K;
      t.abytes = (int64_t)t.mvalid * a.K;
      t.b = (const char*)a.B + (t.e * wrows + t.n0) * a.K;
      t.bbytes = (wrows - t.n0) * a.K;
      slot += per_xcd;
      return true;
    }
    return false;
  };

  // loads of a pair of stages: 8 rows of 128 bytes per wave instruction, chunks swizzled as km2_off reads them
  constexpr int NI = kTile / (kThreads / 8);
  // gate/up: 32 rows of the tile are 16 gate rows and the 16 up rows of the same columns, so that a lane's sums
  // of one block hold both
  auto brow = [&](int r) { return !GU ? r : r / 32 * 16 + (r % 32 < 16 ? r % 32 : a.N + r % 32 - 16); };
  uint32_t va[NI], vb[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = 8 * (wave * NI + i) + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
    va[i] = (uint32_t)(r * a.K) + 16u * c;
    vb[i] = (uint32_t)((int64_t)brow(r) * a.K) + 16u * c;
  }
  const uint32_t rl = lds_addr(ring);
  auto issue = [&](const I8Tile& t, bool any, int pair, uint32_t at) {
    const auto ra = make_rsrc(t.a, any ? t.abytes : 0), rb = make_rsrc(t.b, any ? t.bbytes : 0);
    const uint32_t l0 = at + (uint32_t)(wave * NI * 1024);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(uintptr_t)(l0 + i * 1024), 16, (int)va[i], pair * 2 * kRowB, 0, 0);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void_t*)(uintptr_t)(l0 + S::kSlotA + i * 1024), 16, (int)vb[i], pair * 2 * kRowB, 0, 0);
  };

  // A tile's scales, one per thread, through LDS: held per lane they would take 36 registers
  auto issue_scales = [&](const I8Tile& t, int buf) {
    if (wave >= 2 * kTile / 64) return;
    const uint32_t l0 = lds_addr(scales[0]) + (uint32_t)(buf * (2 * kTile * 4) + wave * 256);
    const int wrows = GU ? 2 * a.N : a.N;
    const bool rows = wave < kTile / 64;
    const auto r = rows ? make_rsrc(a.scale_a + t.r0, (int64_t)t.mvalid * 4)
                        : make_rsrc(a.scale_b + (int64_t)t.e * wrows + t.n0, (int64_t)(wrows - t.n0) * 4);
    const int at = rows ? tid : brow(tid - kTile);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(uintptr_t)l0, 4, 4 * at, 0, 0, 0);
  };

  // Loads run kAhead pairs ahead of the products: a tile's last kAhead pairs load the next tile's first ones, or
  // with fewer pairs those of several tiles. `ld` is the tile after the one that the products have reached (with
  // fewer pairs one further on), ldp its next pair and ldt its number; behind the last tile the loads are of
  // nothing, so that their count stays.
  constexpr int kAhead = kSlots - 1;
  const int nks = a.K / 64, np = (nks + 1) / 2;
  I8Tile cur, ld;
  int slot = blockIdx.x / 8, lslot = slot, ldp = 0, ldt = 0;
  bool some = find(ld, lslot);
  if (!some) return;
  auto next_ld = [&] {
    ldp = 0;
    ldt = (ldt + 1) % kSlots;
    I8Tile t;
    if (some) some = find(t, lslot);
    if (some) ld = t;
  };
  auto issue_ld = [&](int into) {
    if (ldp == 0 && some) issue_scales(ld, ldt);
    issue(ld, some, ldp, rl + (uint32_t)(into * S::kSlot));
  };
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) {
    issue_ld(i);
    if (++ldp == np) next_ld();
  }
  const int arow0 = wm * (kTile / 2), brow0 = wn * 32 * kNN;
  const int inside = max(0, np - kAhead);  // pairs whose loads are of the same tile
  int buf = 0, tbuf = 0;
  bool first = true;
  while (find(cur, slot)) {
    if (inside > 0) next_ld();  // (it was at pair kAhead of this tile)
    acc_t<kElI8> acc[kMN][kNN];
#pragma unroll
    for (int tm = 0; tm < kMN; ++tm)
#pragma unroll
      for (int tn = 0; tn < kNN; ++tn)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[tm][tn][q] = 0;
    // One pair of stages; the loads fill the slot that every wave has read before this pair's barrier. Loads and
    // stores complete in order: of what is younger than this pair's loads, at least the later pairs' loads and, at
    // the head of a tile, the last tile's stores are still on their way.
    auto kloop = [&](auto tma) {
      constexpr int TMA = decltype(tma)::value, kLater = (kSlots - 2) * 2 * NI;
      auto head = [&](int p, const char*& st, uint32_t& fill) {
        if (p < kAhead && !first) wait_vm<kLater + S::kStores>();
        else wait_vm<kLater>();
        __builtin_amdgcn_s_barrier();
        st = ring + buf * S::kSlot;
        fill = rl + (uint32_t)((buf == 0 ? kAhead : buf - 1) * S::kSlot);
        buf = buf == kAhead ? 0 : buf + 1;
      };
      const char* st;
      uint32_t fill;
      for (int p = 0; p < inside; ++p) {
        head(p, st, fill);
        stage_mma<kElI8, false, false, kTile, kTile, kMN, kNN, TMA, 2 * NI, 0>(
            st, st + S::kSlotA, arow0, brow0, lane, acc, [&] { issue(cur, true, p + kAhead, fill); });
        stage_mma<kElI8, false, false, kTile, kTile, kMN, kNN, TMA, 0, 1>(st, st + S::kSlotA, arow0, brow0, lane, acc, [] {});
      }
#pragma unroll 1
      for (int p = inside; p < np; ++p) {
        head(p, st, fill);
        if (ldp == 0 && some) issue_scales(ld, ldt);
        stage_mma<kElI8, false, false, kTile, kTile, kMN, kNN, TMA, 2 * NI, 0>(
            st, st + S::kSlotA, arow0, brow0, lane, acc, [&] { issue(ld, some, ldp, fill); });
        if (2 * p + 1 < nks)
          stage_mma<kElI8, false, false, kTile, kTile, kMN, kNN, TMA, 0, 1>(st, st + S::kSlotA, arow0, brow0, lane, acc, [] {});
        if (++ldp == np) next_ld();
      }
    };
    const int blocks = __builtin_amdgcn_readfirstlane(max(0, min(kMN, (cur.mvalid - arow0 + 31) / 32)));
    if (kMN == 4 && blocks == 4) kloop(std::integral_constant<int, kMN == 4 ? 4 : 0>());
    else if (kMN == 4 && blocks == 3) kloop(std::integral_constant<int, kMN == 4 ? 3 : 0>());
    else if (kMN >= 2 && blocks == 2) kloop(std::integral_constant<int, kMN >= 2 ? 2 : 0>());
    else if (blocks == 1) kloop(std::integral_constant<int, 1>());
    else kloop(std::integral_constant<int, 0>());
    first = false;
    // out: lane l holds row l & 31 of a block and columns 8 g + 4 (l >> 5) .. + 3 of its group g
    const int col0 = wn * (OUTN / kWN);  // the wave's first output column in the tile
    const int nvalid = min(OUTN, a.N - cur.n0);
    float sa[4];  // (those past the wave's blocks are not used)
    f32x4_t sb[4 * kNN];
    const uint32_t at = lds_addr(scales[0]) + (uint32_t)(tbuf * (2 * kTile * 4));
    tbuf = (tbuf + 1) % kSlots;
    read_scales(at + 4 * (arow0 + out_row(lane)), at + 4 * (kTile + brow0 + 4 * (lane >> 5)), sa, sb);
    constexpr int ES = GU ? 4 : 2;
    const int64_t ld = (int64_t)a.N * ES;
    const auto rc = make_rsrc((char*)a.C + cur.r0 * ld + (int64_t)cur.n0 * ES, (cur.mvalid - 1) * ld + (int64_t)nvalid * ES);
#pragma unroll
    for (int tm = 0; tm < kMN; ++tm) {
      const int m = arow0 + tm * 32 + out_row(lane);
      const uint32_t row = (uint32_t)(m * ld);
      if constexpr (GU) {
#pragma unroll
        for (int tn = 0; tn < kNN; ++tn)
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            f32x4_t h;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float gv = (float)acc[tm][tn][4 * g + q] * (sa[tm] * sb[4 * tn + g][q]);
              const float uv = (float)acc[tm][tn][8 + 4 * g + q] * (sa[tm] * sb[4 * tn + 2 + g][q]);
              h[q] = gv * sigmoidf_(gv) * uv;
            }
            const int c = col0 + 16 * tn + out_col(g, lane);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, h), rc, c < nvalid ? (int)(row + 4 * c) : kOutside, 0, 0);
          }
      } else {
#pragma unroll
        for (int tn = 0; tn < kNN; ++tn)
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            uint2 p[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float sum = (float)acc[tm][tn][4 * (g + k) + q];
                v[q] = (OUT == kDown8 ? kYdUnit * sum : sum) * (sa[tm] * sb[4 * tn + g + k][q]);
              }
              p[k] = OUT == kDown8 ? make_uint2(pack_yd(v[0], v[1]), pack_yd(v[2], v[3])) : pack4(v[0], v[1], v[2], v[3]);
            }
            // the halves' lanes exchange: lanes 0..31 get all 8 columns of group g, lanes 32..63 of g + 1
            const auto x = __builtin_amdgcn_permlane32_swap(p[0].x, p[1].x, false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(p[0].y, p[1].y, false, false);
            const u32x4_t o{x[0], y[0], x[1], y[1]};
            const int c = col0 + tn * 32 + 8 * (g + (lane >> 5));
            __builtin_amdgcn_raw_buffer_store_b128(o, rc, c < nvalid ? (int)(row + 2 * c) : kOutside, 0, 0);
          }
      }
    }
  }
  wait_vm<0>();  // the last loads (of nothing) still write zeros to this workgroup's LDS
}

template <int OUT, int TILE>
hipError_t run_i8_tiles(const char* name, const I8Args& a, int64_t tiles, hipStream_t s) {
  auto k = i8_gemm_kernel<OUT, TILE>;
  hipError_t e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, I8Shape<TILE>::kRing);
  if (e != hipSuccess) return e;
  if (tiles <= 0) return hipSuccess;
  // (large and small tiles are shared out to the XCDs apart, each with up to 7 places over)
  const int64_t grid = persistent_grid(tiles + 14);
  {
    MOE_TRACE(name, s);
    MOE_LAUNCH(k, dim3((unsigned)grid), dim3(I8Shape<TILE>::kThreads), I8Shape<TILE>::kRing, s, a);
  }
  return hipGetLastError();
}

// usual: rows of one group on average
template <int OUT>
hipError_t run_i8(const char* name, const I8Args& a, int64_t usual, hipStream_t s) {
  // per chunk at most floor(P_c / tile) + El row tiles; the device-side count decides the work. Of groups of uneven
  // length every second or so has a row tile more than the average fills.
  const int64_t uneven = a.offsets ? 1 : 0;
  auto tiles = [&](int64_t tile, bool bound) {
    const int64_t outn = OUT == kGateUp8 ? tile / 2 : tile;
    const int64_t mt = bound ? a.P_c / tile + a.El : a.El * ((usual + uneven * (tile / 2) + tile - 1) / tile);
    return a.nc * mt * ((a.N + outn - 1) / outn);
  };
  const int64_t cus = cu_count();
  auto rounds = [&](int64_t tile) { return (tiles(tile, false) + cus - 1) / cus; };
  // A round of large tiles takes two to three times as long as one of small ones (the same once they leave CUs
  // idle): 2000 rows x 4096 on 4096 columns 49 (one round) against 47 us (two), 3000 rows 52 (one) against 69
  // (three), 336 rows x 6848 on 2848 columns 66 against 31 us (one of each).
  // A round of tiny tiles takes about 0.65 of one of small ones: 518 rows x 5568 on 448 columns 15 (one round) against
  // 23 us (one), 336 rows x 6848 on 2848 columns 33 (two) against 31 us (one).
  if (rounds(64) <= rounds(128)) return run_i8_tiles<OUT, kTiny>(name, a, tiles(64, true), s);
  if (rounds(128) <= 2 * rounds(256)) return run_i8_tiles<OUT, kSmall>(name, a, tiles(128, true), s);
  return run_i8_tiles<OUT, kLarge>(name, a, tiles(256, true), s);
}

}  // namespace
}  // namespace gg

// Gate/up with exact int32 sums, dequantised by s_row * s_col, SwiGLU -> h (FP32 rows at the start of the h
// buffer: it is quantised per row next, and a BF16 rounding before that would move codes by whole steps);
// h quantised per row (codes after the FP32 values); down -> yd.
hipError_t launch_expert_fwd_i8(const void* xd, const float* xd_scale, const void* w1, const float* w1_scale,
                                const void* w2, const float* w2_scale, const int32_t* offsets, void* h,
                                float* h_scale, void* yd, int H, int I, int El, int c0, int nc, int64_t P_c,
                                int64_t P, int64_t usual, hipStream_t s) {
  if (nc <= 0 || El <= 0) return hipSuccess;
  int8_t* hq = (int8_t*)h + P * (int64_t)I * 4;
  gg::I8Args a{(const int8_t*)xd, xd_scale, (const int8_t*)w1, w1_scale, h, H, I, offsets, El, c0, nc, P_c};
  hipError_t e = gg::run_i8<gg::kGateUp8>("gemm_gateup_swiglu_i8", a, usual, s);
  if (e != hipSuccess) return e;
  e = launch_quantize_h_i8((const float*)h, hq, h_scale, offsets, El, c0, nc, P_c, I, s);
  if (e != hipSuccess) return e;
  gg::I8Args b{hq, h_scale, (const int8_t*)w2, w2_scale, yd, I, H, offsets, El, c0, nc, P_c};
  return gg::run_i8<gg::kDown8>("gemm_down_i8", b, usual, s);
}

// y = dequantised x w^T for the rows of each group (moe_expert_matmul_i8).
hipError_t launch_expert_matmul_i8(int groups, int64_t rows, int N, int K, const void* x, const float* x_scale,
                                   const void* w, const float* w_scale, const int32_t* offsets, void* y,
                                   hipStream_t s) {
  if (groups <= 0 || rows <= 0) return hipSuccess;
  gg::I8Args a{(const int8_t*)x, x_scale, (const int8_t*)w, w_scale, y, K, N, offsets, groups, 0, 1, rows};
  return gg::run_i8<gg::kProduct>("gemm_matmul_i8", a, (rows + groups - 1) / groups, s);
}

}  // namespace moe
