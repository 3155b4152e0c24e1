// Routing by scores: softmax or sigmoid of the logits, a balance bias and groups of experts in the choice, gates from
// the chosen scores; the gradient to the logits; the bias update.
//
//   s = sigmoid(l) or softmax(l), c = RN32(s + b) with s in FP64; the topk_groups groups with the largest sums of
//   their group_top largest c are eligible, the k largest c of their experts are chosen (ties: lower index);
//   gate_j = scale s_j, divided by the sum of the chosen s where they are renormalised.
//
// A choice hangs on the last bit of c, so c is defined by FP64 scores, rounded once: two programs, or two kernels,
// that follow the formula choose the same experts. FP64 exponentials for every logit would take several times the time of
// reading it, though, and nearly every choice is clear without them: choose() selects by FP32 scores whose error has a
// bound. Where two neighbours in the order are nearer than that (one token of 2000), their exact c puts the chosen
// experts and the first one left out in order; where two groups are (one of 25000), or the last one chosen and what is behind
// the first one left out, or two keys are one, the token's wave goes through choose_exact(). (All of these together took 17
// of 86 us at 131072 tokens of 256 experts while all went there and took every expert's exact c: one such wave late in the
// launch holds up its end.)
//
// 16 lanes hold a token's row in registers (4 tokens per wave, float4 loads), and arithmetic bounds the kernel, not HBM. Per
// lane the row's share becomes a sorted list of its five largest: a score's FP32 bits, the last few of which give way to the
// number of the element, so that one insertion is five medians of three and no index travels beside the score. (131072
// tokens of 256 experts in 8 groups: 52 us, 134 MB of logits; 735 vector instructions a wave, about 40 us of issue.) k + 2
// rounds of a maximum over the 16 lanes (DPP) pop the chosen experts and the first two left out. Where a lane's five are used
// up (one token of 600 in groups, of 1200 without), the lists are made again from what is left.
#include <algorithm>

#include "common.h"
#include "launch.h"
#include "route_keys.h"
#include "trace.h"

namespace moe {

constexpr float kMaxFloat = 3.402823466e38f, kLeast = -3e38f;
// NaN counts as -inf, +inf as the largest finite value: a median of three with a NaN is the smallest of the others. (The
// compiler takes a median with the constant -inf for a minimum, which a NaN would leave at the other constant.)
MOE_DEV float clean_logit(float x) {
  float low = -__builtin_huge_valf();
  asm("" : "+v"(low));
  return __builtin_amdgcn_fmed3f(x, low, kMaxFloat);
}
// exp(x) for x <= 0 within 2^-22 of itself (0 below 2^-126): the hardware's exp2 of the rounded product, and the product's
// rounding put back, which plain exp2(x log2 e) would carry |x| times
MOE_DEV float exp_neg(float x) {
  constexpr float kL = 1.44269504088896341f, kLow = 1.92596299112661746887e-8f, kLn2 = 0.693147180559945309f;
  x = fmaxf(x, -200.f);
  const float t = x * kL;
  const float r = __builtin_fmaf(x, kLow, __builtin_fmaf(x, kL, -t));
  return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(r, kLn2, 1.f);
}

// A token's row of logits: a scalar address for the workgroup and 32 bits for the lane's token. False without a token.
struct Row {
  const float* base;
  uint32_t at;  // bytes
  bool live;
  MOE_DEV explicit operator bool() const { return live; }
  MOE_DEV const float* place(int e) const { return (const float*)((const char*)base + (at + 4u * (uint32_t)e)); }
  MOE_DEV float operator[](int e) const { return *place(e); }
};

struct ScoreArgs {
  int softmax, groups, keep, top, renorm;
  float scale;
  int gs;          // experts of a group
  uint32_t magic;  // 2^20 / gs + 1
};
// route_layout's outputs, for a chunk that fits one workgroup; counts null: left to route_layout
struct LayoutArgs {
  int32_t *counts, *offsets, *row_of, *src_token;
  int64_t P_c;
  int e0, El;
};

// Reductions over the 16 lanes of a token: DPP within a row of 16 (neighbours, pairs, mirrored halves, mirrored row).
template <int CTRL> MOE_DEV int dpp_i(int x) { return __builtin_amdgcn_mov_dpp(x, CTRL, 0xf, 0xf, true); }
template <int CTRL> MOE_DEV float dpp_f(float x) { return __int_as_float(dpp_i<CTRL>(__float_as_int(x))); }
template <int CTRL> MOE_DEV uint32_t dpp_u(uint32_t x) { return (uint32_t)dpp_i<CTRL>((int)x); }
template <int CTRL> MOE_DEV double dpp_d(double x) {
  return __hiloint2double(dpp_i<CTRL>(__double2hiint(x)), dpp_i<CTRL>(__double2loint(x)));
}
#define MOE_ROW16(x, op, get)                              \
  x = op(x, get<0xB1>(x)); x = op(x, get<0x4E>(x));        \
  x = op(x, get<0x141>(x)); x = op(x, get<0x140>(x))
MOE_DEV float add_f(float a, float b) { return a + b; }
MOE_DEV double add_d(double a, double b) { return a + b; }
MOE_DEV uint32_t or_u(uint32_t a, uint32_t b) { return a | b; }
MOE_DEV uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }
MOE_DEV uint32_t min_u(uint32_t a, uint32_t b) { return a < b ? a : b; }
MOE_DEV float row_min(float x) { MOE_ROW16(x, fminf, dpp_f); return x; }
MOE_DEV float row_sum(float x) { MOE_ROW16(x, add_f, dpp_f); return x; }
MOE_DEV double row_sum_d(double x) { MOE_ROW16(x, add_d, dpp_d); return x; }
MOE_DEV uint32_t row_or(uint32_t x) { MOE_ROW16(x, or_u, dpp_u); return x; }
MOE_DEV uint32_t row_max_u(uint32_t x) { MOE_ROW16(x, max_u, dpp_u); return x; }
MOE_DEV uint32_t row_min_u(uint32_t x) { MOE_ROW16(x, min_u, dpp_u); return x; }

// (HIP's own take an int, which the compiler makes of a condition, and a condition of that.)
MOE_DEV uint64_t ballot(bool x) { return __builtin_amdgcn_ballot_w64(x); }
MOE_DEV bool any_lane(bool x) { return ballot(x) != 0; }

// LDS between lanes of one wave: program order, which the compiler has to keep.
MOE_DEV void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); __builtin_amdgcn_wave_barrier(); }

constexpr int kSelInts = 2 * kGroup;  // LDS of a token: its groups' keys, then its slots (key and lane, one slot per lane)

// Group of expert e, without a division: e < 1024, so floor(e / gs) = (e (2^20 / gs + 1)) >> 20 (ScoreArgs::magic).
MOE_DEV int group_of(int e, uint32_t magic) { return (int)(((uint32_t)e * magic) >> 20); }

// A median of three is also a maximum, one that leaves its operands as they are (fmaxf first makes them canonical; the
// compiler takes a median with the constant +inf for fmaxf).
MOE_DEV float plain_max(float a, float b) {
  float high = __builtin_huge_valf();
  asm("" : "+v"(high));
  return __builtin_amdgcn_fmed3f(a, b, high);
}
MOE_DEV float row_max(float x) { MOE_ROW16(x, plain_max, dpp_f); return x; }
MOE_DEV void two_largest(float& b0, float& b1, float x) {
  b1 = __builtin_amdgcn_fmed3f(b0, b1, x);
  b0 = plain_max(b0, x);
}

// Softmax: the row's largest logit and FP64 sum of exponentials (0 where no logit is above -inf).
MOE_DEV double exact_sum(const Row& row, int E, int q, float& m) {
  const float ninf = -__builtin_huge_valf();
  m = ninf;
  if (row)
#pragma unroll 4
    for (int e = q; e < E; e += kGroup) m = fmaxf(m, clean_logit(row[e]));
  m = row_max(m);
  double den = 0.0;
  if (row && m > ninf)
#pragma unroll 2
    for (int e = q; e < E; e += kGroup) den += exp((double)clean_logit(row[e]) - (double)m);
  return row_sum_d(den);
}
MOE_DEV float exact_c(float logit, const float* bias, int e, bool softmax, float m, double den) {
  const double l = clean_logit(logit);
  const double s = !softmax ? 1.0 / (1.0 + exp(-l)) : den > 0.0 ? exp(l - (double)m) / den : 0.0;
  const float x = (float)(bias ? s + (double)bias[e] : s);
  return x != x ? -__builtin_huge_valf() : x;
}

// The eligible groups of a token, one bit each, from the c of its experts in LDS. P lanes share a group (16 of them with
// up to one group, 1 with nine or more), and lane q has the groups q / P, q / P + 16 / P, ... Lane q's float4s are
// q nv .. q nv + nv - 1, so that with nv a
// power of two the lanes start at different ones of the 16 that the banks hold. near: whether the last eligible
// and the first other group are within `margin` (relative to 1 or the largest c that any group adds), where c is not
// exact; two groups with one sum are near.
// cut (where a token of the wave has near groups): what no c that a group adds is below. keys: LDS of the token, kSelInts.
template <bool EXACT>
MOE_DEV uint64_t eligible_groups(const float* c, uint32_t* keys, int q, const ScoreArgs& a, float margin, bool& near, float& cut) {
  const int gs = a.gs;
  const float ninf = -__builtin_huge_valf();
  int lp = 0;  // log2 P: whole float4 per lane, and no more lanes than there are for the groups
  while (lp < 4 && (a.groups << (lp + 1)) <= kGroup && gs % (8 << lp) == 0) ++lp;
  const int P = 1 << lp, part = q & (P - 1), first = q >> lp, per_pass = kGroup >> lp;
  float mine[4], size = 1.f;
  cut = __builtin_huge_valf();
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int g = first + per_pass * u;
    mine[u] = ninf;
    if (per_pass * u >= a.groups) continue;
    float b0 = ninf, b1 = ninf;
    if (g < a.groups) {
      if ((gs & 3) == 0) {
        const int nv = gs >> (2 + lp);
        const float4* p = (const float4*)(c + g * gs) + part * nv;
        const int start = nv & (nv - 1) ? 0 : (q * min(nv, 16)) >> 4;
        for (int n = 0; n < nv; ++n) {
          const float4 x = p[n ^ start];
          two_largest(b0, b1, x.x); two_largest(b0, b1, x.y); two_largest(b0, b1, x.z); two_largest(b0, b1, x.w);
        }
      } else {
        for (int e = g * gs; e < (g + 1) * gs; ++e) two_largest(b0, b1, c[e]);
      }
    }
#define MOE_STEP(CTRL) { const float o0 = dpp_f<CTRL>(b0), o1 = dpp_f<CTRL>(b1); two_largest(b0, b1, o0); two_largest(b0, b1, o1); }
    if (lp > 0) MOE_STEP(0xB1)
    if (lp > 1) MOE_STEP(0x4E)
    if (lp > 2) MOE_STEP(0x141)
    if (lp > 3) MOE_STEP(0x140)
#undef MOE_STEP
    if (g < a.groups) {
      const bool two = a.top == 2 && gs > 1;
      mine[u] = two ? b0 + b1 : b0;
      size = fmaxf(size, two ? fmaxf(fabsf(b0), fabsf(b1)) : fabsf(b0));
      cut = fminf(cut, two ? b1 : b0);
    }
  }
  uint32_t lo = 0, hi = 0, least = ~0u, most = 0;
  // up to 32 groups' keys go through LDS, four to a load (0 behind the last), instead of a shuffle each (131072 tokens, 8
  // groups: 75 -> 73.5 us)
  const bool few = a.groups <= kSelInts;
  if (few) {
    keys[q] = 0;
    keys[q + kGroup] = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int g = first + per_pass * u;
      if (per_pass * u < a.groups && g < a.groups) keys[g] = EXACT ? logit_key(mine[u]) : ordered(mine[u]);
    }
    wave_lds_fence();
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int g = first + per_pass * u;
    if (per_pass * u >= a.groups) continue;
    int beaten = 0;
    const uint32_t own = EXACT ? logit_key(mine[u]) : ordered(mine[u]);
    auto meet = [&](uint32_t other, int o) {
      if constexpr (EXACT) beaten += other > own || (other == own && o < g);
      else beaten += other > own;
    };
    if (few) {
      for (int o = 0; o < a.groups; o += 4) {
        const uint4 k = *(const uint4*)(keys + o);
        meet(k.x, o); meet(k.y, o + 1); meet(k.z, o + 2); meet(k.w, o + 3);
      }
    } else {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t key = EXACT ? logit_key(mine[w]) : ordered(mine[w]);
        const int count = min(kGroup, a.groups - kGroup * w);  // (more than 32 groups: one lane each)
        for (int j = 0; j < count; ++j) meet((uint32_t)__shfl((int)key, j, kGroup), kGroup * w + j);
      }
    }
    if (g < a.groups) {
      if (beaten < a.keep) {
        if (g < 32) lo |= 1u << g; else hi |= 1u << (g - 32);
        least = min(least, own);
      } else {
        most = max(most, own);
      }
    }
  }
  lo = row_or(lo);
  hi = a.groups > 32 ? row_or(hi) : 0;
  if constexpr (!EXACT) {
    least = row_min_u(least);
    most = row_max_u(most);
    size = __uint_as_float(row_max_u(__float_as_uint(size)));  // (not negative)
    near = !(key_logit(least) - key_logit(most) > margin * size) || __popc(lo) + __popc(hi) != a.keep;
    if (any_lane(near)) cut = row_min(cut) - margin * size;
  }
  return ((uint64_t)hi << 32) | lo;
}

// Slots in the order of their experts' exact c, ties to the lower expert: lane j < n brings slot j's expert, and takes the
// one whose place j is. Every lane of the wave calls.
MOE_DEV int order_exact(const Row& row, const float* bias, uint32_t* slots, int id, int E, int n, int q, const ScoreArgs& a) {
  float m = 0.f;
  const double den = a.softmax ? exact_sum(row, E, q, m) : 0.0;
  const bool live = row && q < n;
  const uint32_t key = live ? logit_key(exact_c(row[id], bias, id, a.softmax, m, den)) : 0u;
  int place = 0;
  for (int j = 0; j < n; ++j) {
    const uint32_t other = (uint32_t)__shfl((int)key, j, kGroup);
    const int other_id = __shfl(id, j, kGroup);
    place += other > key || (other == key && other_id < id);
  }
  wave_lds_fence();
  if (live) slots[place] = (uint32_t)id;
  wave_lds_fence();
  return live ? (int)slots[q] : 0;
}

// The choice where the FP32 sums do not tell: lane j < k returns slot j's expert. c: the token's row in LDS [E], FP32 sums;
// those not below `cut` are made exact, and the choice is among them. regroup: the eligible groups are chosen again (the row
// holds every group's sums; otherwise the eligible ones', and lower values). Every lane of the wave calls.
MOE_DEV int choose_exact(const Row& row, const float* bias, float* c, uint32_t* slots, int E, int K, int q,
                         const ScoreArgs& a, float cut, bool regroup) {
  float m = 0.f;
  const double den = a.softmax ? exact_sum(row, E, q, m) : 0.0;
  uint64_t mine = 0;  // of this lane's experts q, q + 16, ...
#pragma unroll 4
  for (int i = 0; i < 64; ++i) {
    const int e = kGroup * i + q;
    if (kGroup * i >= E) break;
    if (e < E && c[e] >= cut) mine |= 1ull << i;
  }
  for (uint64_t u = row ? mine : 0; any_lane(u != 0); u &= u - 1) {
    if (u) {
      const int e = kGroup * (__ffsll((unsigned long long)u) - 1) + q;
      c[e] = exact_c(row[e], bias, e, a.softmax, m, den);
    }
  }
  wave_lds_fence();
  if (regroup) {
    bool unused;
    float none;
    const uint64_t open = eligible_groups<true>(c, slots, q, a, 0.f, unused, none);
    uint64_t kept = 0;
    for (uint64_t u = mine; u; u &= u - 1) {
      const int i = __ffsll((unsigned long long)u) - 1;
      if ((open >> (group_of(kGroup * i + q, a.magic) & 63)) & 1) kept |= 1ull << i;
    }
    mine = kept;
  }
  int id = 0;
  for (int s = 0; s < K; ++s) {
    // the lane's largest, the first of equal ones; then the row's, and of equal ones the lowest expert
    uint32_t top = 0, at = 0;
    for (uint64_t u = mine; u; u &= u - 1) {
      const uint32_t e = (uint32_t)(kGroup * (__ffsll((unsigned long long)u) - 1) + q);
      const uint32_t key = logit_key(c[e]);
      at = key > top ? e : at;
      top = key > top ? key : top;
    }
    const uint32_t best = row_max_u(top);
    const uint32_t e = 1023u - row_max_u(top == best && best ? 1023u - at : 0u);
    if (q == s) id = min((int)e, E - 1);
    if (q == (int)(e & (kGroup - 1))) mine &= ~(1ull << (e / kGroup));
  }
  return id;
}

constexpr int kTopList = 5;  // a lane's list

// Experts of a lane's elements: VEC: 64 (i / 4) + 4 q + i % 4 (float4 loads, E a multiple of 4), else 16 i + q.
template <bool VEC> MOE_DEV int expert_of(int i, int q) { return VEC ? 64 * (i / 4) + 4 * q + i % 4 : kGroup * i + q; }
template <int NE, bool VEC>
MOE_DEV void load_row(const Row& row, int E, int q, float none, float (&x)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; i += VEC ? 4 : 1) {
    const int e = expert_of<VEC>(i, q);
    if constexpr (VEC) {
      float4 f = make_float4(none, none, none, none);
      if (row && e < E) f = *(const float4*)row.place(e);
      x[i] = f.x; x[i + 1] = f.y; x[i + 2] = f.z; x[i + 3] = f.w;
    } else {
      x[i] = row && e < E ? row[e] : none;
    }
  }
}

// A row of 16 NE floats in LDS, whole: no lane asks which of its elements there are.
template <int NE, bool VEC>
MOE_DEV void load_lds(const float* row, int q, float (&x)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; i += VEC ? 4 : 1) {
    const float* p = row + expert_of<VEC>(i, q);
    if constexpr (VEC) {
      const float4 f = *(const float4*)p;
      x[i] = f.x; x[i + 1] = f.y; x[i + 2] = f.z; x[i + 3] = f.w;
    } else {
      x[i] = *p;
    }
  }
}

// The choice of a token's 16 lanes: lane j < k returns slot j's expert. row: its logits, null without a token; c: its row in
// LDS [16 NE]; x: the row in registers; b_row: the bias in LDS [16 NE], kLeast .. kMaxFloat (NaN: kLeast), and what keeps
// the places behind the last expert out (-kMaxFloat); slots: its kSelInts in LDS. Every lane of the wave calls.
//
// Error of the FP32 sums, in units of 2^-24: sigmoid: the exponential's argument and its own ulp move s by at most 0.72 (s
// (1 - s) |l| <= 0.224), 1 + e rounds by 1 and the reciprocal by 2, the sum with the bias by |c|, and the exact c
// itself by |c|: 3.72 + 2 |c| each, so that sums further apart than 2 (3.72 + 2 |c|) < 16 max(1, |c|) are in order.
// Softmax: the differences and products below an exponential move it by 2.2 x e^-x <= 0.82, its ulp by 2, relative to a
// largest score p = 1 / sum; the sum (in FP64) by its terms' 3, the reciprocal and the product by 3: 9 p + 2 |c| each.
// That is a bound for sums: keys, whose last bits hold an element's number, lie up to NE - 1 steps (2 (NE - 1) units of
// a sum's size) from theirs on either side, so that they only say which sums to look at. Sums within the margin, ties
// among them, go to order_exact or, where they are not all among the slots, to choose_exact.
// m, inv: softmax: the row's largest logit and 1 / the sum of exponentials (0 where no logit is above -inf).
template <int NE, bool VEC>
MOE_DEV int choose(const Row& row, float (&x)[NE], const float* bias, const float* b_row, float* c, uint32_t* slots, int E,
                   int K, int q, const ScoreArgs& a, float& m, float& inv) {
  const float ninf = -__builtin_huge_valf();
  constexpr float kLog2e = 1.44269504088896341f, kUnit = 0x1p-24f;
  constexpr float none = -kMaxFloat;  // no expert: below kLeast, the lowest score
  const float margin = (a.softmax ? 20.f : 16.f) * kUnit;  // relative to the sums and, softmax, p, or 1
  m = ninf;
  inv = 0.f;
  if (a.softmax) {
#pragma unroll
    for (int i = 0; i < NE; ++i) { x[i] = clean_logit(x[i]); m = fmaxf(m, x[i]); }
    m = row_max(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      x[i] = m > ninf ? __builtin_amdgcn_exp2f((x[i] - m) * kLog2e) : 0.f;
      sum += (double)x[i];
    }
    const float total = (float)row_sum_d(sum);
    inv = total > 0.f ? __builtin_amdgcn_rcpf(total) : 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) x[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i)  // (the median costs no instruction, and takes 0 for NaN)
      x[i] = __builtin_amdgcn_fmed3f(__builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x[i] * kLog2e)), 0.f, 1.f);
  }
  {
    float b[NE];
    load_lds<NE, VEC>(b_row, q, b);
#pragma unroll
    for (int i = 0; i < NE; ++i) x[i] += b[i];
  }
  // the sums in LDS: for the groups, and for choose_exact
  auto store_sums = [&]() {
#pragma unroll
    for (int i = 0; i < NE; i += VEC ? 4 : 1) {
      float* p = c + expert_of<VEC>(i, q);
      if constexpr (VEC) *(float4*)p = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      else *p = x[i];
    }
    wave_lds_fence();
  };
  bool regroup = false, exact = false;
  float cut = kLeast;  // of choose_exact: every eligible expert
  if (a.keep < a.groups) {
    store_sums();
    bool near;
    float low;
    // twice the margin of one c and the sums' rounding, relative to 1 (softmax scores are at most that)
    const uint64_t open = eligible_groups<false>(c, slots, q, a, 2.f * margin + 4.f * kUnit, near, low);
    regroup = any_lane(row && near);
    if (a.keep * (a.top == 2 && a.gs > 1 ? 2 : 1) >= K) cut = fmaxf(low, kLeast);  // the eligible groups add k that are not below it
    if (!regroup) {  // the others' sums give way in LDS
      if (VEC && (a.gs & 3) == 0) {  // the four of a vector share a group
#pragma unroll
        for (int i = 0; i < NE; i += 4) {
          const int e = expert_of<VEC>(i, q);
          if (!((open >> (group_of(e, a.magic) & 63)) & 1)) *(float4*)(c + e) = make_float4(none, none, none, none);
        }
      } else {
        for (int e = q; e < E; e += kGroup)
          if (!((open >> group_of(e, a.magic)) & 1)) c[e] = none;
      }
      wave_lds_fence();
      load_lds<NE, VEC>(c, q, x);
    }
  } else {
    store_sums();
  }
  int id = 0;
  if (!regroup) {
    constexpr uint32_t kNumber = NE - 1;  // the bits that hold an element's number
    constexpr uint32_t kUnknown = 0xffffffffu;
    uint32_t key[kTopList];
    // The list: the five largest, sorted, as keys that order as the scores. again: of those below `limit`.
    auto make_list = [&](bool again, float limit) {
      float l[kTopList];
#pragma unroll
      for (int j = 0; j < kTopList; ++j) l[j] = none;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        float v = __uint_as_float((__float_as_uint(x[i]) & ~kNumber) | i);
        if (again) v = v < limit ? v : none;
#pragma unroll
        for (int j = kTopList - 1; j > 0; --j) l[j] = __builtin_amdgcn_fmed3f(l[j - 1], l[j], v);
        l[0] = plain_max(l[0], v);
      }
#pragma unroll
      for (int j = 0; j < kTopList; ++j) key[j] = ordered(l[j]);
    };
    // Rounds s0 .. rounds - 1. After a lane's fifth its next is unknown where it had more.
    const int rounds = min(K + 2, a.keep * a.gs);  // the slots, and the first two experts left out where there are
    const int tokens = __popcll(ballot(row.live)) / kGroup;  // of this wave
    auto play = [&](int s0) {
      int pops = 0;
      for (int s = s0; s < rounds; ++s) {
        const uint32_t best = row_max_u(key[0]);
        const bool pop = key[0] == best;
        pops += __popcll(ballot(row && pop));
        if (pop) {
          *(uint2*)(slots + 2 * s) = make_uint2(best, (uint32_t)q);
#pragma unroll
          for (int j = 0; j + 1 < kTopList; ++j) key[j] = key[j + 1];
          key[kTopList - 1] = NE > kTopList ? kUnknown : 0u;
        }
      }
      wave_lds_fence();
      // two lanes of one token with one key popped both: more pops than rounds
      return pops != (rounds - s0) * tokens;
    };
    make_list(false, 0.f);
    bool twins = play(0);
    uint2 mine = *(const uint2*)(slots + 2 * q);
    if constexpr (NE > kTopList) {
      while (!twins && any_lane(row && q < rounds && mine.x == kUnknown)) {
        // From the first unknown slot of the wave's tokens on, with what each lane has left below its last. (Of twins a
        // slot holds one only: the other's lane could not tell what it has left.)
        const uint64_t unknown = ballot(row && q < rounds && mine.x == kUnknown);
        int s0 = rounds;
        for (uint64_t u = unknown; u; u &= u - 1) s0 = min(s0, (int)(__ffsll((unsigned long long)u) - 1) & (kGroup - 1));
        uint32_t last = kUnknown;
        for (int s = 0; s < s0; ++s) last = slots[2 * s + 1] == (uint32_t)q ? slots[2 * s] : last;
        load_lds<NE, VEC>(c, q, x);
        make_list(true, last == kUnknown ? __builtin_huge_valf() : key_logit(last));
        wave_lds_fence();
        twins |= play(s0);
        mine = *(const uint2*)(slots + 2 * q);
      }
    }
    const uint32_t bits = mine.x >> 31 ? mine.x : ~mine.x;  // (of a negative score the key holds the complement)
    const int i = (int)(bits & kNumber);
    id = VEC ? 64 * (i / 4) + 4 * (int)mine.y + i % 4 : kGroup * i + (int)mine.y;
    // The keys propose an order, and the sums in LDS tell whether it holds: slots 0 .. K are clear of each other where each
    // sum is above the next by more than the margin (a sum below the next one, which its number put in front, is not).
    const float mine_c = q < rounds ? c[id] : 0.f;
    const float next_c = dpp_f<0x101>(mine_c);  // of lane q + 1
    auto above = [&](float u, float v) {
      const float size = fmaxf(fabsf(u), fabsf(v));
      return u - v > margin * (a.softmax ? inv + size : fmaxf(1.f, size)) + 0x1p-100f;
    };
    const bool near = q < K && q + 1 < rounds && !above(mine_c, next_c);
    // No expert behind slot K has a key above slot K + 1's, so none has a sum above all that share that key but for the
    // number. The K slots in front are clear of these, or the choice is not among slots 0 .. K.
    bool more = false;
    if (rounds > K + 1) {
      const float least = row_min(q < K ? mine_c : __builtin_huge_valf());
      more = !above(least, key_logit(slots[2 * (K + 1)] | kNumber));
    }
    exact = twins || any_lane(row && more);
    if (exact) {
      // What is not below the last one popped, with room for its error: at least as many were popped as there are rounds.
      // (Twins pop more than one a round: the last slot may hold no expert, or a NaN where a list ran out, and then every
      // eligible one is looked at.)
      const float v = key_logit(slots[2 * (rounds - 1)]);
      cut = fmaxf(v - 64.f * (margin + 2 * NE * kUnit) * fmaxf(1.f, fabsf(v)), kLeast);
    } else if (any_lane(row && near)) {
      id = order_exact(row, bias, slots, id, E, min(K + 1, rounds), q, a);
    }
  }
  if (regroup || exact) id = choose_exact(row, bias, c, slots, E, K, q, a, cut, regroup);
  return id;
}

// Gate of lane j < k (live) for its expert; m and inv as choose() leaves them.
MOE_DEV float gate_of(const Row& row, int id, bool live, float m, float inv, const ScoreArgs& a) {
  const float ninf = -__builtin_huge_valf();
  const float z = live ? clean_logit(row[id]) : ninf;
  float g;
  if (a.renorm) {
    // relative to the largest chosen score: a sum of very small ones keeps its digits
    const float low = a.softmax ? z : fminf(z, 0.f);
    const float top = row_max(low);
    float u = 0.f;
    if (live && top > ninf) u = a.softmax ? exp_neg(z - top) : exp_neg(low - top) * __builtin_amdgcn_rcpf(1.f + exp_neg(-fabsf(z)));
    const float sum = row_sum(u);
    g = sum > 0.f ? u * __builtin_amdgcn_rcpf(sum) : 0.f;
  } else if (a.softmax) {
    g = live && m > ninf ? exp_neg(z - m) * inv : 0.f;
  } else {
    g = exp_neg(fminf(z, 0.f)) * __builtin_amdgcn_rcpf(1.f + exp_neg(-fabsf(z)));
  }
  return a.scale * g;
}

// Where a chunk fits one workgroup: its counts, offsets, rows and the rows' tokens, as route_layout leaves them, from the
// histogram of its tokens and the lanes' own expert (lane q < k of a token's 16; live).
template <int THREADS>
MOE_DEV void layout_chunk(const int* hist, int* space, const LayoutArgs& o, int id, bool live, int64_t t0, int tl, int q,
                          int E, int K, int ch) {
  const int tid = threadIdx.x, El = o.El;
  uint64_t* mask = (uint64_t*)space;  // [El] the tokens that chose a local expert
  int* off = space + 2 * El;          // [El + 1]
  for (int e = tid; e < E; e += THREADS) o.counts[(int64_t)ch * E + e] = hist[e];
  for (int el = tid; el < El; el += THREADS) mask[el] = 0;
  if (tid < 64) {
    int run = 0;
    for (int b = 0; b < El; b += 64) {
      const int v = b + tid < El ? hist[o.e0 + b + tid] : 0;
      int incl = v;
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) {
        const int u = __shfl_up(incl, s, 64);
        if (tid >= s) incl += u;
      }
      if (b + tid < El) off[b + tid] = run + incl - v;
      run += __shfl(incl, 63, 64);
    }
    if (tid == 0) off[El] = run;
  }
  __syncthreads();
  for (int el = tid; el <= El; el += THREADS) o.offsets[(int64_t)ch * (El + 1) + el] = off[el];
  const int el = id - o.e0;
  const bool local = live && el >= 0 && el < El;
  if (local) atomicOr((unsigned long long*)&mask[el], 1ull << tl);
  __syncthreads();
  if (live) {
    int32_t row = -1;
    if (local) {
      const uint64_t below = tl == 0 ? 0ull : ~0ull >> (64 - tl);
      const int64_t r = (int64_t)ch * o.P_c + off[el] + __popcll(mask[el] & below);
      o.src_token[r] = (int32_t)(t0 + tl);
      row = (int32_t)r;
    }
    o.row_of[(t0 + tl) * K + q] = row;
  }
  for (int64_t r = off[El] + tid; r < o.P_c; r += THREADS) o.src_token[(int64_t)ch * o.P_c + r] = -1;
}

// THREADS / 16 tokens per workgroup: 64 (one histogram per layout block: its four 16-token places take the sum and
// zeros, one 16-byte store) or, where 64 rows of LDS are too many, 16. Waves without a token leave the choice out.
template <int NE, bool VEC, int THREADS>
__global__ __launch_bounds__(THREADS, THREADS == 1024 && VEC ? 8 : 1) void route_scores_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias, int32_t* __restrict__ topk_idx,
    float* __restrict__ gates, int32_t* __restrict__ block_hist, int64_t T, int64_t tc, int E, int K, int chunk0, ScoreArgs a,
    LayoutArgs o) {
  extern __shared__ __attribute__((aligned(16))) int smem[];  // slots, histogram [E4], bias [16 NE], c [tokens][16 NE]
  constexpr int kTok = THREADS / kGroup;
  const int E4 = (E + 3) & ~3;
  int* hist = smem + kTok * kSelInts;
  const int tid = threadIdx.x, q = tid & (kGroup - 1), tl = tid / kGroup;
  uint32_t* slots = (uint32_t*)smem + tl * kSelInts;
  float* b_row = (float*)(hist + E4);
  float* c = b_row + kGroup * NE * (1 + tl);
  const int ch = chunk0 + blockIdx.y, bl = blockIdx.x, nbpc = gridDim.x;
  const int64_t t0 = ch * tc + (int64_t)bl * kTok;
  const bool valid = tl < (int)min(min(T, (ch + 1) * tc) - t0, (int64_t)kTok);
  const Row row{logits + t0 * E, 4u * (uint32_t)(tl * E), valid};
  const bool live = valid && q < K;
  float x[NE];
  load_row<NE, VEC>(row, E, q, -__builtin_huge_valf(), x);
  for (int e = tid; e < kGroup * NE; e += THREADS) {
    if (e < E) hist[e] = 0;
    b_row[e] = e >= E ? -kMaxFloat : bias ? __builtin_amdgcn_fmed3f(bias[e], kLeast, kMaxFloat) : 0.f;
  }
  __syncthreads();
  int id = 0;
  if (any_lane(valid)) {
    float m, inv;
    id = choose<NE, VEC>(row, x, bias, b_row, c, slots, E, K, q, a, m, inv);
    const float g = gate_of(row, id, live, m, inv, a);
    if (live) {
      topk_idx[t0 * K + (tl * K + q)] = id;
      gates[t0 * K + (tl * K + q)] = g;
      atomicAdd(&hist[id], 1);
    }
  }
  __syncthreads();
  if (o.counts) {
    layout_chunk<THREADS>(hist, (int*)(hist + E4), o, id, live, t0, tl, q, E, K, ch);
    return;
  }
  // expert-major: the counts of an expert over the chunk's histograms lie one behind the other
  if constexpr (THREADS == 1024) {
    int4* out = (int4*)block_hist + (int64_t)ch * E * nbpc + bl;
    for (int e = tid; e < E; e += THREADS) out[(int64_t)e * nbpc] = make_int4(hist[e], 0, 0, 0);
  } else {
    int32_t* out = block_hist + (int64_t)ch * E * nbpc + bl;
    for (int e = tid; e < E; e += THREADS) out[(int64_t)e * nbpc] = hist[e];
  }
}

// Gradient to the logits. With gh_j = s_j / sum s over the chosen experts:
//   sigmoid: dl_j = scale gh_j (1 - s_j)(dg_j - sum gh_i dg_i), or scale s_j (1 - s_j) dg_j where gates are not renormalised
//   softmax: dl_j = scale gh_j (dg_j - sum gh_i dg_i), or, for every expert, scale p_e ([e = idx_j] dg_j - sum p_i dg_i)
// 1 - s_j is taken as sigmoid(-l_j). Bound by HBM: the row of E gradients is written, read too where every logit has one.
// 16 lanes per token, as in the forward; a row of LDS per token, cleared by its lanes, takes the k values to their
// places, so that each row leaves in float4 stores. ADD: dlogits holds another term. The planes are route_bwd_dlogits'.
template <int NE, bool VEC, bool DENSE, bool ADD>
__global__ __launch_bounds__(256) void route_scores_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ dgates, const int32_t* __restrict__ idx,
    float* __restrict__ dlogits, uint16_t* __restrict__ dl_hi, uint16_t* __restrict__ dl_lo, int ldl, int64_t pitch,
    int64_t t0, int64_t t1, int K, int E, ScoreArgs a) {
  extern __shared__ __attribute__((aligned(16))) int smem[];  // [16 tokens][16 NE]
  const int tid = threadIdx.x, q = tid & (kGroup - 1), tl = tid / kGroup;
  float* d_row = (float*)smem + tl * (kGroup * NE);
  const int64_t tb = t0 + (int64_t)blockIdx.x * kHistTok, t = tb + tl;
  const bool valid = t < t1;
  const float ninf = -__builtin_huge_valf();
  const Row lr{logits + tb * E, 4u * (uint32_t)(tl * E), valid};
  const bool live = valid && q < K;
  const int id = live ? idx[t * K + q] : 0;
  const float d = live ? dgates[t * K + q] : 0.f;
  float p[DENSE ? NE : 1];
  if constexpr (DENSE) load_row<NE, VEC>(lr, E, q, ninf, p);
  const float z = live ? clean_logit(lr[id]) : ninf;
#pragma unroll
  for (int i = 0; i < NE; i += 4) *(float4*)(d_row + 16 * i + 4 * q) = make_float4(0.f, 0.f, 0.f, 0.f);
  float v, mean = 0.f;
  if constexpr (DENSE) {
    float m = ninf, s = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) { p[i] = clean_logit(p[i]); m = fmaxf(m, p[i]); }
    m = row_max(m);
#pragma unroll
    for (int i = 0; i < NE; ++i) { p[i] = m > ninf ? expf(p[i] - m) : 0.f; s += p[i]; }
    s = row_sum(s);
    const float inv = s > 0.f ? 1.f / s : 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) p[i] *= inv;
    const float pj = live && m > ninf ? expf(z - m) * inv : 0.f;
    mean = -a.scale * row_sum(pj * d);
    v = a.scale * pj * d;
  } else if (a.renorm) {
    const float low = a.softmax ? z : fminf(z, 0.f);
    const float top = row_max(low);
    float u = 0.f;
    if (live && top > ninf) u = a.softmax ? expf(z - top) : expf(low - top) / (1.f + expf(-fabsf(z)));
    const float s = row_sum(u);
    const float gh = s > 0.f ? u / s : 0.f;
    const float rest = a.softmax ? 1.f : expf(-fmaxf(z, 0.f)) / (1.f + expf(-fabsf(z)));
    v = a.scale * gh * rest * (d - row_sum(gh * d));
  } else {
    const float e1 = expf(-fabsf(z));
    v = a.scale * d * e1 / ((1.f + e1) * (1.f + e1));  // s (1 - s)
  }
  wave_lds_fence();
  if (live) d_row[id] = v;
  wave_lds_fence();
  if (!valid) return;
  float* row = dlogits + t * (int64_t)E;
#pragma unroll
  for (int i = 0; i < NE; i += VEC ? 4 : 1) {
    const int e = expert_of<VEC>(i, q);
    if constexpr (VEC) {
      float4 f = *(const float4*)(d_row + e);
      if constexpr (DENSE) {
        f.x += mean * p[i]; f.y += mean * p[i + 1]; f.z += mean * p[i + 2]; f.w += mean * p[i + 3];
      }
      if (e < E) {
        if constexpr (ADD) {
          const float4 o = *(const float4*)(row + e);
          f.x += o.x; f.y += o.y; f.z += o.z; f.w += o.w;
        }
        *(float4*)(row + e) = f;
      }
      if (dl_hi && e < ldl) {  // zeros past E
        const uint32_t h0 = pack_bf2(f.x, f.y), h1 = pack_bf2(f.z, f.w);
        *(uint2*)(dl_hi + (t - t0) * pitch + e) = make_uint2(h0, h1);
        *(uint2*)(dl_lo + (t - t0) * pitch + e) = make_uint2(pack_bf2(f.x - bf2f(h0 & 0xffff), f.y - bf2f(h0 >> 16)),
                                                             pack_bf2(f.z - bf2f(h1 & 0xffff), f.w - bf2f(h1 >> 16)));
      }
    } else if (e < E) {
      float f = d_row[e];
      if constexpr (DENSE) f += mean * p[i];
      if constexpr (ADD) f += row[e];
      row[e] = f;
    }
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

static ScoreArgs score_args(const moe_router_scores& r, int E) {
  const int gs = E / r.n_groups;
  return {r.score == MOE_SCORE_SOFTMAX, r.n_groups, r.topk_groups, r.group_top, r.renormalize != 0, r.scale, gs,
          (1u << 20) / (uint32_t)gs + 1};
}

// Elements per lane: the row's experts over 16 lanes, 4, 8, ... 64.
static int elements_per_lane(int E) {
  int ne = 4;
  while (ne * kGroup < E) ne *= 2;
  return ne;
}
#define MOE_NE(E, VECTOR, CALL)                              \
  do {                                                       \
    if ((VECTOR)) {                                          \
      constexpr bool VEC = true;                             \
      switch (elements_per_lane(E)) {                        \
        case 4: { constexpr int NE = 4; CALL; break; }       \
        case 8: { constexpr int NE = 8; CALL; break; }       \
        case 16: { constexpr int NE = 16; CALL; break; }     \
        case 32: { constexpr int NE = 32; CALL; break; }     \
        default: { constexpr int NE = 64; CALL; }            \
      }                                                      \
    } else {                                                 \
      constexpr bool VEC = false;                            \
      switch (elements_per_lane(E)) {                        \
        case 4: { constexpr int NE = 4; CALL; break; }       \
        case 8: { constexpr int NE = 8; CALL; break; }       \
        case 16: { constexpr int NE = 16; CALL; break; }     \
        case 32: { constexpr int NE = 32; CALL; break; }     \
        default: { constexpr int NE = 64; CALL; }            \
      }                                                      \
    }                                                        \
  } while (0)
// float4 loads need rows that start at 16 bytes
static bool vector_rows(int E, const void* a, const void* b) { return E % 4 == 0 && (((uintptr_t)a | (uintptr_t)b) & 15) == 0; }

template <typename Kernel>
static hipError_t allow_lds(Kernel k, size_t bytes) {
  return bytes > 65536 ? hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)
                       : hipSuccess;
}

hipError_t launch_route_scores(const moe_router_scores& r, const float* logits, const float* bias, int32_t* topk_idx,
                               float* gates, int32_t* counts, int32_t* offsets, int32_t* row_of, int32_t* src_token,
                               int32_t* scratch, int64_t T, int E, int e0, int El, int K, int n, int chunk0, int nchunks,
                               int64_t P_c, hipStream_t s) {
  const int blocks = route_blocks_per_chunk(T, n);
  const int64_t tc = (T + n - 1) / n;
  const ScoreArgs a = score_args(r, E);
  // 64 tokens per workgroup keep the histograms few and let a chunk of up to 64 tokens be one workgroup; 16 where 64 rows
  // of c would leave a CU one workgroup, and where there are too few tokens for every CU: their waves, one per SIMD,
  // then finish earlier. (256 experts, launches one behind the other in a graph, 16 against 64: 256 tokens 13.2 and
  // 14.7 us, 8192 15.0 and 16.6, 16384 17.1 and 16.8, 131072 in two chunks 61.7 and 58.8.)
  const bool wide = E <= 256 && tc > kHistTok && (tc <= 64 || T > 8192);
  const int tok = wide ? 64 : kHistTok;
  const int nbpc = wide ? blocks : blocks * kSub;
  const bool whole = tc <= tok;  // a chunk is one workgroup
  LayoutArgs o{};
  if (whole) o = LayoutArgs{counts, offsets, row_of, src_token, P_c, e0, El};
  const size_t lds = (size_t)(tok * kSelInts + (E + 3) / 4 * 4 + (tok + 1) * kGroup * elements_per_lane(E)) * 4;
  hipError_t err = hipSuccess;
  {
    MOE_TRACE("route_scores", s);
#define MOE_RS(THREADS)                                                                                             \
    {                                                                                                               \
      auto k = route_scores_kernel<NE, VEC, THREADS>;                                                               \
      err = allow_lds(k, lds);                                                                                      \
      for (int ch = 0; ch < nchunks && err == hipSuccess; ch += 65535) { /* chunks of a launch: the grid's y */     \
        MOE_LAUNCH(k, dim3(whole ? 1 : nbpc, std::min(nchunks - ch, 65535)), dim3(THREADS), lds, s, logits, bias,   \
                   topk_idx, gates, scratch, T, tc, E, K, chunk0 + ch, a, o);                                       \
        err = hipGetLastError();                                                                                    \
      }                                                                                                             \
    }
    const bool vec = vector_rows(E, logits, bias);
    MOE_NE(E, vec, if constexpr (NE <= 16) { if (wide) MOE_RS(1024) else MOE_RS(256) } else { MOE_RS(256) });
#undef MOE_RS
  }
  if (err != hipSuccess || whole) return err;
  return launch_layout(topk_idx, scratch, counts, offsets, row_of, src_token, T, E, e0, El, K, n, chunk0, nchunks, P_c, s);
}

hipError_t launch_route_scores_bwd(const moe_router_scores& r, const float* logits, const float* dgates,
                                   const int32_t* idx, float* dlogits, int64_t t0, int64_t t1, int K, int E,
                                   hipStream_t s, uint16_t* dl_hi, uint16_t* dl_lo, int ldl, int64_t pitch, bool add) {
  const bool vec = vector_rows(E, logits, dlogits);
  const int width = dl_hi && ldl > E ? ldl : E;  // columns that a lane's elements have to reach
  const int ne = elements_per_lane(width);
  if (dl_hi && (!vec || !dl_lo || ldl < E || ldl > ne * kGroup || ldl % 4 || pitch % 4 || pitch < ldl)) return hipErrorInvalidValue;
  if (t1 <= t0) return hipSuccess;
  const ScoreArgs a = score_args(r, E);
  const bool dense = a.softmax && !a.renorm;
  const size_t lds = (size_t)kHistTok * kGroup * ne * 4;
  MOE_TRACE("route_scores_bwd", s);
#define MOE_RSB(DENSE, ADD)                                                                                            \
  MOE_LAUNCH((route_scores_bwd_kernel<NE, VEC, DENSE, ADD>), dim3((unsigned)((t1 - t0 + kHistTok - 1) / kHistTok)),    \
             dim3(256), lds, s, logits, dgates, idx, dlogits, dl_hi, dl_lo, ldl, pitch, t0, t1, K, E, a)
  MOE_NE(width, vec, if (dense && add) MOE_RSB(true, true); else if (dense) MOE_RSB(true, false);
         else if (add) MOE_RSB(false, true); else MOE_RSB(false, false));
#undef MOE_RSB
  return hipGetLastError();
}

hipError_t launch_router_bias_update(int E, int rows, const int32_t* counts, float rate, float* bias, hipStream_t s) {
  MOE_TRACE("router_bias_update", s);
  MOE_LAUNCH(router_bias_update_kernel, dim3(1), dim3(256), 0, s, E, rows, counts, rate, bias);
  return hipGetLastError();
}

}  // namespace moe
