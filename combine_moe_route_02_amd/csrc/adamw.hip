// AdamW over many tensors at once, with moving averages in FP32 or in 8 bits, and the norm of their gradients.
//
//   g = grad * grad_scale, m' = b1 m + (1 - b1) g, v' = b2 v + (1 - b2) g^2,
//   w' = w (1 - lr wd) - lr / (1 - b1^t) * m' / (sqrt(v' / (1 - b2^t)) + eps)
//
// Bound by HBM: 28 bytes per parameter with a BF16 gradient, an FP32 master and FP32 averages (gradient 2, master 8,
// averages 16, BF16 weight 2), 16 with averages in 8 bits. A wave owns a block of 256 elements that share a scale, four
// in a row per lane, so that each FP32 access is 1 KiB without gaps and the block's largest value and scale are scalars;
// two blocks per wave keep enough loads in flight. A workgroup takes tiles of 2048 elements; the tensors of a launch
// and the tile each starts at are kernel arguments, so no table travels to the device.
//
// 8-bit averages. m = s c|c| / 127^2 and v = s c^4 / 255^4 with s the block's largest magnitude: the steps grow with
// the value, so that entries 10^-4 (m) or 10^-9 (v) of the block's largest keep digits, which equal steps would lose.
// A step of training moves m and v by some per cent or less, under half a code, and rounding to the nearest code
// would hold them where they are; so the code above is taken with the chance of how near it is (by 16 bits: the expected value
// is off by 2^-16 of a step of the codes at most), by a hash of the element's place, the step and the seed. v > 0 never rounds to 0: m / sqrt(v) stays bounded.
// Every FP32 operation that decides a code is rounded once (no contraction), so the codes are defined bit by bit.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "trace.h"

#pragma clang fp contract(off)

namespace moe {

constexpr int kAdamThreads = 256;
constexpr int kAdamBlock = 256;                      // elements per scale of an 8-bit average: four per lane of a wave
constexpr int kAdamTile = kAdamThreads / 64 * 2 * kAdamBlock;  // elements per workgroup
constexpr int kAdamFew = 40, kAdamMany = 256;         // tensors per launch: arguments of 3.4 and 21 KiB

struct AdamTensor {
  void* w;
  float* master;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  uint32_t place;   // of element 0 in the random sequence (low 32 bits)
  float lr_scale, wd;
};
template <int N>
struct AdamBatch {
  uint32_t tile0[N];  // first tile of each tensor in this launch, ascending (empty tensors are left out)
  int count;
  AdamTensor t[N];
};
struct AdamConst {
  double lr, beta1, beta2, eps;
  double unbias1, unbias2;  // 1 / (1 - b1^step), 1 / sqrt(1 - b2^step); from *step_dev on the device where it is given
  const double* lr_dev;
  const int64_t* step_dev;
  const float* grad_scale;
  int64_t step;
  uint32_t seed;
};

// The tensor of a tile: the last one whose first tile is not behind it. One lane per tensor: kernel arguments may lie in host
// memory, where the six dependent loads of a binary search took longer than the rest of a small launch
// (97 tensors: 38 -> 20 us with this and one launch for three).
template <int N>
MOE_DEV int tensor_of(const AdamBatch<N>& b, uint32_t tile) {
  const int lane = threadIdx.x & 63;
  int before = 0;
#pragma unroll
  for (int i = 0; i < N; i += 64) {
    const int at = i + lane;
    before += __popcll(__ballot(at < b.count && b.tile0[at < N ? at : 0] <= tile));
  }
  return __builtin_amdgcn_readfirstlane(before - 1);
}

// Random bits of an element: three 16-bit numbers, for m, v and a BF16 weight. Odd multipliers from the digits of the
// golden ratio, e and pi; shifts carry the high bits down.
MOE_DEV uint32_t step_key(uint32_t seed, int64_t step) {
  uint32_t k = (uint32_t)step * 0x243F6A89u + seed;
  k ^= k >> 16;
  k *= 0xB7E15163u;
  return k ^ (k >> 15);
}
MOE_DEV uint32_t random_bits(uint32_t place, uint32_t key, int j) {  // of element place + j
  uint32_t x = place * 0x9E3779B9u + key + (uint32_t)j * 0x9E3779B9u;
  x = (x ^ (x >> 16)) * 0xB7E15163u;
  return x ^ (x >> 15);
}
MOE_DEV uint32_t more_bits(uint32_t x) { return (x * 0x243F6A89u) >> 16; }

// Values of codes in units of the block's scale.
constexpr float kInv127 = (float)(1.0 / 127.0), kInv255 = (float)(1.0 / 255.0);
MOE_DEV float level_m(float c) { const float t = c * kInv127; return t * t; }
MOE_DEV float level_v(float c) { float t = c * kInv255; t = t * t; return t * t; }
MOE_DEV float decode_m(int8_t code, float scale) {
  const float t = (float)code * kInv127;
  return t * fabsf(t) * scale;
}
MOE_DEV float decode_v(uint8_t code, float scale) { return level_v((float)code) * scale; }

// Code of a in [0, 1], as a float: the level below, or the one above where (a - below) / (above - below) exceeds r. The root
// only proposes the level below (it is off by far less than one); a neighbour takes its place where a lies outside. The last
// level is 1 exactly, so the code above it is never taken.
template <bool FOURTH>
MOE_DEV float encode(float a, float r) {
  auto level = [](float c) { return FOURTH ? level_v(c) : level_m(c); };
  float root = __builtin_amdgcn_sqrtf(a);
  if (FOURTH) root = __builtin_amdgcn_sqrtf(root);
  float c = floorf(root * (FOURTH ? 255.f : 127.f));
  float lo = level(c), hi = level(c + 1.f), d = a - lo, w = hi - lo;
  if (__float_as_uint(d) >= __float_as_uint(w)) {  // below 0 (the sign) or not below w: of 64 lanes seldom one
    c += a < lo ? -1.f : a >= hi ? 1.f : 0.f;
    lo = level(c);
    d = a - lo;
    w = level(c + 1.f) - lo;
  }
  return c + (d > r * w ? 1.f : 0.f);
}

// Largest magnitude over the wave, by bits (NaN above infinity above every number): DPP within rows of 16, then scalars.
template <int CTRL>
MOE_DEV uint32_t dpp_max(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xf, 0xf, true));
}
MOE_DEV float block_max(uint32_t bits) {
  bits = dpp_max<0xB1>(bits);   // neighbours, pairs, mirrored halves, mirrored row
  bits = dpp_max<0x4E>(bits);
  bits = dpp_max<0x141>(bits);
  bits = dpp_max<0x140>(bits);
  const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)bits, 0), (uint32_t)__builtin_amdgcn_readlane((int)bits, 16));
  const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)bits, 32), (uint32_t)__builtin_amdgcn_readlane((int)bits, 48));
  return __uint_as_float(max(a, b));
}
// Blocks whose largest value is under 2^-120 count as zeros: its reciprocal would leave the range. An infinite one
// has no codes: the block becomes NaN, as with a NaN.
MOE_DEV float block_scale(float big) {
  return big < 0x1p-120f ? 0.f : big == __builtin_huge_valf() ? __builtin_nanf("") : big;
}
MOE_DEV float block_inv(float scale) { return scale > 0.f ? 1.0f / scale : 0.f; }
MOE_DEV float share(float x, float inv) {
  return fminf(fabsf(x) * inv, 1.0f);  // never NaN (infinity times 0 gives 1: the scale is NaN then)
}

// A tile: its elements are addressed by a scalar pointer and 32 bits per lane, half the registers of 64-bit addresses.
template <typename T> MOE_DEV T* at(T* p, int i) { return (T*)((char*)p + (uint32_t)i * (uint32_t)sizeof(T)); }
template <typename T> MOE_DEV const T* at(const T* p, int i) { return (const T*)((const char*)p + (uint32_t)i * (uint32_t)sizeof(T)); }

// Four elements from i on, of a tile of n: vectors inside, single ones at its end. Loads and stores are nontemporal: a step
// reads each value once, and what it writes is read again a step later at the earliest. (75.8 million parameters with the
// norm before it: 467 us -> 428 by the stores, 427 -> 359 by the loads, which leave the gradients of the norm in the cache.
// The norm's own loads are plain, and the codes' too: nontemporal ones took 204 us instead of 215 with 8-bit averages, but
// reading the codes next 124 instead of 106.)
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
// Loads leave the bits as they are: a conversion beside its load would wait for it, and so for every load before the next.
template <typename T> struct Raw;
template <> struct Raw<float> {
  f32x4_t x;
  MOE_DEV void values(float* f) const { f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w; }
};
template <> struct Raw<uint16_t> {
  u32x2_t x;
  MOE_DEV void values(float* f) const {
    f[0] = bf2f(x.x & 0xffff); f[1] = bf2f(x.x >> 16); f[2] = bf2f(x.y & 0xffff); f[3] = bf2f(x.y >> 16);
  }
};
MOE_DEV Raw<float> load4(const float* p, int i, int n) {
  if (i + 4 <= n) return {__builtin_nontemporal_load((const f32x4_t*)at(p, i))};
  float f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = i + j < n ? *at(p, i + j) : 0.f;
  return {f32x4_t{f[0], f[1], f[2], f[3]}};
}
MOE_DEV Raw<uint16_t> load4(const uint16_t* p, int i, int n) {
  if (i + 4 <= n) return {__builtin_nontemporal_load((const u32x2_t*)at(p, i))};
  uint32_t f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = i + j < n ? *at(p, i + j) : 0u;
  return {u32x2_t{f[0] | (f[1] << 16), f[2] | (f[3] << 16)}};
}
template <typename T>
MOE_DEV void store4(T* p, int i, int n, const float* f) {
  if (i + 4 <= n) {
    if constexpr (sizeof(T) == 2)
      __builtin_nontemporal_store(u32x2_t{pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3])}, (u32x2_t*)at(p, i));
    else
      __builtin_nontemporal_store(f32x4_t{f[0], f[1], f[2], f[3]}, (f32x4_t*)at(p, i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) if (i + j < n) st_elem(at(p, i + j), f[j]);
  }
}
MOE_DEV uint32_t load_codes(const uint8_t* p, int i, int n) {
  if (i + 4 <= n) return *(const uint32_t*)at(p, i);
  uint32_t c = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) if (i + j < n) c |= (uint32_t)*at(p, i + j) << (8 * j);
  return c;
}
MOE_DEV void store_codes(uint8_t* p, int i, int n, uint32_t c) {
  if (i + 4 <= n) {
    __builtin_nontemporal_store(c, (uint32_t*)at(p, i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) if (i + j < n) *at(p, i + j) = (uint8_t)(c >> (8 * j));
  }
}
MOE_DEV void decode4(uint32_t mc, uint32_t vc, float ms, float vs, float* m, float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[j] = decode_m((int8_t)(mc >> (8 * j)), ms);
    v[j] = decode_v((uint8_t)(vc >> (8 * j)), vs);
  }
}

// A lane's four values to codes; a block's scales are stored by its first lane. NEAREST: r is 1/2.
template <bool NEAREST>
MOE_DEV void pack4(const float* m, const float* v, const uint32_t* rnd, int i, int n, uint8_t* mc, float* ms,
                   uint8_t* vc, float* vs) {
  uint32_t bm = 0, bv = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    bm = max(bm, __float_as_uint(m[j]) & 0x7fffffffu);
    bv = max(bv, __float_as_uint(v[j]) & (NEAREST ? 0x7fffffffu : ~0u));  // (a step's v': no sign but a NaN's)
  }
  bv &= 0x7fffffffu;
  const float sm = block_scale(block_max(bm)), sv = block_scale(block_max(bv));
  const float im = block_inv(sm), iv = block_inv(sv);
  uint32_t cm[4], cv = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float rm = NEAREST ? 0.5f : (float)(rnd[j] & 0xffffu) * 0x1p-16f;
    const float rv = NEAREST ? 0.5f : (float)(rnd[j] >> 16) * 0x1p-16f;
    cm[j] = (uint32_t)(int)copysignf(encode<false>(share(m[j], im), rm), m[j]);  // (a NaN's code does not matter)
    const float a = share(v[j], iv);
    cv = __builtin_amdgcn_cvt_pk_u8_f32(fmaxf(encode<true>(a, rv), ceilf(a)), j, cv);  // (a > 0: 1 at least)
  }
  if (i < n) {
    const uint32_t low = __builtin_amdgcn_perm(cm[1], cm[0], 0x0c0c0400u), high = __builtin_amdgcn_perm(cm[3], cm[2], 0x0c0c0400u);
    store_codes(mc, i, n, low | (high << 16));
    store_codes(vc, i, n, cv);
    if (i % kAdamBlock == 0) { *at(ms, i / kAdamBlock) = sm; *at(vs, i / kAdamBlock) = sv; }
  }
}
// First element of a lane's four in block u (0, 1) of its wave, in a tile.
MOE_DEV int lane_element(int u) { return (int)(threadIdx.x >> 6) * 2 * kAdamBlock + u * kAdamBlock + (threadIdx.x & 63) * 4; }
// Elements of a tile.
MOE_DEV int tile_size(int64_t n, int64_t first) { return (int)min(n - first, (int64_t)kAdamTile); }
// The scale of a lane's block, the same for the wave; 0 behind the tensor's end.
MOE_DEV float scale_of(const float* scale, int i, int n) {
  const int block = i / kAdamBlock;
  return block * kAdamBlock < n ? *at(scale, block) : 0.f;
}

// W: float, or uint16_t (BF16 bits) with a master or, without one, rounded by chance like the codes: an update under
// half a step of BF16 (2^-9 of the weight; lr is 10^-4) would otherwise never reach the weight.
template <typename W, bool MASTER, typename G, bool Q8, int N>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(const AdamBatch<N> b, const AdamConst k) {
  const int which = tensor_of(b, blockIdx.x);
  const AdamTensor& t = b.t[which];
  const float gs = k.grad_scale ? *k.grad_scale : 1.0f;
  if (!(fabsf(gs) <= 3.402823466e38f)) return;  // a norm that is not finite: the step is left out
  int64_t step = k.step;
  double unbias1 = k.unbias1, unbias2 = k.unbias2;
  if (k.step_dev) {
    step = max((int64_t)1, *k.step_dev);
    unbias1 = -1.0 / expm1((double)step * log(k.beta1));
    unbias2 = 1.0 / sqrt(-expm1((double)step * log(k.beta2)));
  }
  const double lr = (k.lr_dev ? *k.lr_dev : k.lr) * (double)t.lr_scale;
  const float b1 = (float)k.beta1, o1 = (float)(1.0 - k.beta1), b2 = (float)k.beta2, o2 = (float)(1.0 - k.beta2);
  const float keep = (float)(1.0 - lr * (double)t.wd);
  const float c1 = (float)(lr * unbias1), c2 = (float)unbias2;
  const float eps = (float)k.eps;
  const int64_t first = (int64_t)(blockIdx.x - b.tile0[which]) * kAdamTile;
  const int n = tile_size(t.n, first);
  const G* grad = (const G*)t.grad + first;
  W* weight = (W*)t.w + first;
  float* master = t.master + first;  // (MASTER)
  using State = std::conditional_t<Q8, uint8_t, float>;
  State *m_state = (State*)t.m + first, *v_state = (State*)t.v + first;
  float *m_scale = t.m_scale + first / kAdamBlock, *v_scale = t.v_scale + first / kAdamBlock;  // (Q8)
  const uint32_t place = t.place + (uint32_t)first;
  using Weight = std::conditional_t<MASTER, float, W>;
  Raw<G> g_raw[2];
  Raw<Weight> w_raw[2];
  Raw<float> m_raw[2], v_raw[2];  // FP32 averages
  uint32_t m_code[2], v_code[2];  // 8 bits
  float m_unit[2], v_unit[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane_element(u);
    g_raw[u] = load4(grad, i, n);
    if constexpr (MASTER) w_raw[u] = load4((const float*)master, i, n);
    else w_raw[u] = load4((const W*)weight, i, n);
    if constexpr (Q8) {
      m_code[u] = load_codes(m_state, i, n);
      v_code[u] = load_codes(v_state, i, n);
      m_unit[u] = scale_of(m_scale, i, n);
      v_unit[u] = scale_of(v_scale, i, n);
    } else {
      m_raw[u] = load4((const float*)m_state, i, n);
      v_raw[u] = load4((const float*)v_state, i, n);
    }
  }
  constexpr bool kChance = Q8 || (sizeof(W) == 2 && !MASTER);
  const uint32_t key = kChance ? step_key(k.seed, step) : 0;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane_element(u);
    float g[4], w[4], m[4], v[4];
    g_raw[u].values(g);
    w_raw[u].values(w);
    if constexpr (Q8) {
      decode4(m_code[u], v_code[u], m_unit[u], v_unit[u], m, v);
    } else {
      m_raw[u].values(m);
      v_raw[u].values(v);
    }
    uint32_t rnd[4];
    if constexpr (kChance) {
#pragma unroll
      for (int j = 0; j < 4; ++j) rnd[j] = random_bits(place + (uint32_t)i, key, j);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = g[j] * gs;
      m[j] = m[j] * b1 + x * o1;
      v[j] = v[j] * b2 + (x * x) * o2;
      // the hardware's root and reciprocal, 2^-23 each, beside the 2^-24 of the sum: no state hangs on their bits
      w[j] = w[j] * keep - c1 * m[j] * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(v[j]) * c2 + eps);
    }
    if constexpr (MASTER) store4(master, i, n, w);
    if constexpr (sizeof(W) == 2 && !MASTER) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = __float_as_uint(w[j]);
        if ((x & 0x7f800000u) != 0x7f800000u) w[j] = __uint_as_float((x + more_bits(rnd[j])) & 0xffff0000u);
      }
    }
    store4(weight, i, n, w);
    if constexpr (Q8) {
      pack4<false>(m, v, rnd, i, n, m_state, m_scale, v_state, v_scale);
    } else {
      store4(m_state, i, n, m);
      store4(v_state, i, n, v);
    }
  }
}

// 8-bit averages to FP32 and back (nearest level).
__global__ __launch_bounds__(kAdamThreads) void adamw_unpack_kernel(int64_t size, const uint8_t* __restrict__ mc,
                                                                    const float* __restrict__ ms,
                                                                    const uint8_t* __restrict__ vc,
                                                                    const float* __restrict__ vs,
                                                                    float* __restrict__ m, float* __restrict__ v) {
  const int64_t first = (int64_t)blockIdx.x * kAdamTile;
  const int n = tile_size(size, first);
  mc += first; vc += first; m += first; v += first;
  ms += first / kAdamBlock; vs += first / kAdamBlock;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane_element(u);
    float fm[4], fv[4];
    decode4(load_codes(mc, i, n), load_codes(vc, i, n), scale_of(ms, i, n), scale_of(vs, i, n), fm, fv);
    store4(m, i, n, fm);
    store4(v, i, n, fv);
  }
}

__global__ __launch_bounds__(kAdamThreads) void adamw_pack_kernel(int64_t size, const float* __restrict__ m,
                                                                  const float* __restrict__ v, uint8_t* __restrict__ mc,
                                                                  float* __restrict__ ms, uint8_t* __restrict__ vc,
                                                                  float* __restrict__ vs) {
  const int64_t first = (int64_t)blockIdx.x * kAdamTile;
  const int n = tile_size(size, first);
  mc += first; vc += first; m += first; v += first;
  ms += first / kAdamBlock; vs += first / kAdamBlock;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane_element(u);
    float fm[4], fv[4];
    const Raw<float> rm = load4(m, i, n), rv = load4(v, i, n);
    rm.values(fm);
    rv.values(fv);
    pack4<true>(fm, fv, nullptr, i, n, mc, ms, vc, vs);
  }
}

// Norm of all gradients: FP64 sums of squares, one per workgroup (the workgroups of every launch walk the same tiles
// in the same order, and a later launch adds to the sums of the ones before), then one workgroup adds them. No more
// workgroups than tiles (1105 weights: 12.9 -> 12.0 us for norm and update).
constexpr int kNormBlocks = 2048;
MOE_DEV double wave_sum_d(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}
MOE_DEV double group_sum_d(double x) {  // of a workgroup of kAdamThreads; in thread 0
  __shared__ double part[kAdamThreads / 64];
  x = wave_sum_d(x);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kAdamThreads / 64; ++w) s += part[w];
  return s;
}

// Four 16-byte loads per lane and tile.
constexpr int kNormLoads = 4;
template <typename G> constexpr int kNormVec = 16 / sizeof(G);
template <typename G> constexpr int kNormTile = kAdamThreads * kNormVec<G> * kNormLoads;
template <typename G, int N>
__global__ __launch_bounds__(kAdamThreads) void grad_norm_kernel(const AdamBatch<N> b, uint32_t tiles, int written,
                                                                 double* __restrict__ sums) {
  constexpr int V = kNormVec<G>;
  double s = 0.0;
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += kNormBlocks) {
    const int which = tensor_of(b, tile);
    const G* grad = (const G*)b.t[which].grad;
    const int64_t n = b.t[which].n, i = (int64_t)(tile - b.tile0[which]) * kNormTile<G> + threadIdx.x * V;
    float g[kNormLoads][V];
#pragma unroll
    for (int u = 0; u < kNormLoads; ++u) {
      const int64_t at = i + u * (kAdamThreads * V);
      if (at + V <= n) {
        const u32x4 x = *(const u32x4*)(grad + at);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (V == 8) { g[u][2 * j] = bf2f(w[j] & 0xffff); g[u][2 * j + 1] = bf2f(w[j] >> 16); }
          else g[u][j] = __uint_as_float(w[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) g[u][j] = at + j < n ? ld_elem(grad + at + j) : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kNormLoads; ++u)
      // squares in FP64: those of BF16 values would be exact in FP32's digits, but not within its range
#pragma unroll
      for (int j = 0; j < V; ++j) s = __builtin_fma((double)g[u][j], (double)g[u][j], s);
  }
  s = group_sum_d(s);
  if (threadIdx.x == 0) sums[blockIdx.x] = (int)blockIdx.x < written ? sums[blockIdx.x] + s : s;
}

__global__ __launch_bounds__(kAdamThreads) void grad_norm_total_kernel(const double* __restrict__ sums, int count,
                                                                       double max_norm, float* __restrict__ norm) {
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += kAdamThreads) s += sums[i];
  s = group_sum_d(s);
  if (threadIdx.x == 0) {
    const double x = sqrt(s);
    norm[0] = (float)x;
    // a norm that is no finite FP32 number cannot be scaled by: NaN, which leaves the step out
    norm[1] = !(fabs(x) <= 3.4028234663852886e38) ? __builtin_nanf("") : x > max_norm ? (float)(max_norm / x) : 1.0f;
  }
}

// ------------------------------------------------------------------------------------------------ host

namespace {

int kind_of(const moe_adamw_tensor& t) {
  return (t.w_dtype == MOE_BF16 ? (t.master ? 2 : 4) : 0) + (t.grad_dtype == MOE_BF16 ? 1 : 0);
}

// Runs `launch(batch, tiles)` over the tensors for which `pick` holds, N at a time, in tiles of `tile` elements. Elements are
// placed in the random sequence as if the tensors lay one behind the other in their order, each from a multiple of 256 on.
template <int N, typename Pick, typename Launch>
hipError_t over_batches_of(int n_tensors, const moe_adamw_tensor* t, int64_t tile, Pick pick, Launch launch) {
  AdamBatch<N> b;
  b.count = 0;
  int64_t place = 0, tiles = 0;
  auto flush = [&]() -> hipError_t {
    if (b.count == 0) return hipSuccess;
    const hipError_t e = launch(b, (uint32_t)tiles);
    b.count = 0;
    tiles = 0;
    return e;
  };
  for (int i = 0; i < n_tensors; ++i) {
    const int64_t blocks = (t[i].n + kAdamBlock - 1) / kAdamBlock;
    if (t[i].n > 0 && pick(t[i])) {
      const int64_t mine = (t[i].n + tile - 1) / tile;
      if (b.count == N || tiles + mine > (1 << 23)) {  // a launch holds fewer than 2^32 threads
        const hipError_t e = flush();
        if (e != hipSuccess) return e;
      }
      b.tile0[b.count] = (uint32_t)tiles;
      b.t[b.count++] = AdamTensor{t[i].w, t[i].master, t[i].grad, t[i].m, t[i].v, t[i].m_scale, t[i].v_scale, t[i].n,
                                  (uint32_t)(place * kAdamBlock), t[i].lr_scale, t[i].weight_decay};
      tiles += mine;
    }
    place += blocks;
  }
  return flush();
}
// The launch's arguments are copied whole: few tensors take the short list (100000 weights: 40 tensors 6.0 us, 41 with the
// long list 6.3).
template <typename Pick, typename Launch>
hipError_t over_batches(int n_tensors, const moe_adamw_tensor* t, int64_t tile, Pick pick, Launch launch) {
  return n_tensors <= kAdamFew ? over_batches_of<kAdamFew>(n_tensors, t, tile, pick, launch)
                               : over_batches_of<kAdamMany>(n_tensors, t, tile, pick, launch);
}

template <typename W, bool MASTER, typename G, int N>
hipError_t launch_kind(const AdamBatch<N>& b, uint32_t tiles, const AdamConst& k, bool q8, hipStream_t s) {
  MOE_TRACE("adamw", s);
  if (q8) MOE_LAUNCH((adamw_kernel<W, MASTER, G, true, N>), dim3(tiles), dim3(kAdamThreads), 0, s, b, k);
  else MOE_LAUNCH((adamw_kernel<W, MASTER, G, false, N>), dim3(tiles), dim3(kAdamThreads), 0, s, b, k);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(const moe_adamw_options& o, int n_tensors, const moe_adamw_tensor* t, hipStream_t s) {
  const double step = (double)o.step;
  const AdamConst k{o.lr, o.beta1, o.beta2, o.eps, -1.0 / std::expm1(step * std::log(o.beta1)),
                    1.0 / std::sqrt(-std::expm1(step * std::log(o.beta2))), o.lr_dev, o.step_dev, o.grad_scale, o.step, o.seed};
  const bool q8 = o.state_bits == 8;
  for (int kind = 0; kind < 6; ++kind) {
    const hipError_t e = over_batches(
        n_tensors, t, kAdamTile, [&](const moe_adamw_tensor& x) { return kind_of(x) == kind; },
        [&](const auto& b, uint32_t tiles) {
          switch (kind) {
            case 0: return launch_kind<float, false, float>(b, tiles, k, q8, s);
            case 1: return launch_kind<float, false, uint16_t>(b, tiles, k, q8, s);
            case 2: return launch_kind<uint16_t, true, float>(b, tiles, k, q8, s);
            case 3: return launch_kind<uint16_t, true, uint16_t>(b, tiles, k, q8, s);
            case 4: return launch_kind<uint16_t, false, float>(b, tiles, k, q8, s);
            default: return launch_kind<uint16_t, false, uint16_t>(b, tiles, k, q8, s);
          }
        });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

int64_t grad_norm_ws_bytes() { return kNormBlocks * (int64_t)sizeof(double); }

hipError_t launch_grad_norm(int n_tensors, const moe_adamw_tensor* t, double max_norm, float* norm, void* workspace,
                            hipStream_t s) {
  double* sums = (double*)workspace;
  int count = 0;  // sums that hold something
  for (int bf16 = 0; bf16 < 2; ++bf16) {
    const hipError_t e = over_batches(
        n_tensors, t, bf16 ? kNormTile<uint16_t> : kNormTile<float>, [&](const moe_adamw_tensor& x) { return (x.grad_dtype == MOE_BF16) == (bf16 == 1); },
        [&](const auto& b, uint32_t tiles) {
          constexpr int N = sizeof(b.tile0) / sizeof(uint32_t);
          const int blocks = (int)std::min<uint32_t>(tiles, kNormBlocks), written = count;
          count = std::max(count, blocks);
          MOE_TRACE("grad_norm", s);
          if (bf16) MOE_LAUNCH((grad_norm_kernel<uint16_t, N>), dim3(blocks), dim3(kAdamThreads), 0, s, b, tiles, written, sums);
          else MOE_LAUNCH((grad_norm_kernel<float, N>), dim3(blocks), dim3(kAdamThreads), 0, s, b, tiles, written, sums);
          return hipGetLastError();
        });
    if (e != hipSuccess) return e;
  }
  MOE_TRACE("grad_norm_total", s);
  MOE_LAUNCH(grad_norm_total_kernel, dim3(1), dim3(kAdamThreads), 0, s, sums, count, max_norm, norm);
  return hipGetLastError();
}

hipError_t launch_adamw_unpack(int64_t n, const void* mc, const float* ms, const void* vc, const float* vs, float* m,
                               float* v, hipStream_t s) {
  MOE_TRACE("adamw_unpack", s);
  MOE_LAUNCH(adamw_unpack_kernel, dim3((unsigned)((n + kAdamTile - 1) / kAdamTile)), dim3(kAdamThreads), 0, s, n,
             (const uint8_t*)mc, ms, (const uint8_t*)vc, vs, m, v);
  return hipGetLastError();
}

hipError_t launch_adamw_pack(int64_t n, const float* m, const float* v, void* mc, float* ms, void* vc, float* vs,
                             hipStream_t s) {
  MOE_TRACE("adamw_pack", s);
  MOE_LAUNCH(adamw_pack_kernel, dim3((unsigned)((n + kAdamTile - 1) / kAdamTile)), dim3(kAdamThreads), 0, s, n, m, v,
             (uint8_t*)mc, ms, (uint8_t*)vc, vs);
  return hipGetLastError();
}

}  // namespace moe
