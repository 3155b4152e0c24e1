// Per-row quantisation to 8-bit integers, for the integer expert path: weights and plain activations
// (moe_quantize_rows_i8), token rows on their way into dispatch order (moe_dispatch), and the FP32
// rows of h between the two expert products.
//
// Symmetric codes of one row: scale = amax / 127, code = RNE(v * (127 / amax)) in [-127, 127], both
// with one FP32 rounding per step; a row of zeros has codes 0 and scale 1. A row that holds a NaN or
// an infinity has codes 0 and scale NaN, so what is computed from it is NaN. All are bound by their
// bytes: one wave per row, 16-byte loads, and the row stays in registers between its absmax and its
// codes where it fits (up to 16 vectors a lane), so it is read once. 8192 rows of 7168 values 34 us (5.2 TB/s; 32 to
// 36 from card to card), 16K rows of 768 FP32 values 11.2 us.
#include <algorithm>

#include "common.h"
#include "i8.h"
#include "launch.h"
#include "trace.h"

namespace moe {

constexpr int kI8RowsPerBlock = 4;  // one wave per row
constexpr int kI8MaxVec = 16;       // 16-byte vectors of a row that a lane holds

// Magnitude bits of a row's values, compared as integers: monotone, and NaN ranks above infinity, so
// the maximum also says whether every value is finite.
MOE_DEV uint32_t magnitude8(const u32x4& v) {  // 8 BF16 values, both halves of a word at once
  typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;
  auto half = [](uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7fff7fffu); };
  const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(half(v.x), half(v.y)),
                                            __builtin_elementwise_max(half(v.z), half(v.w)));
  return (uint32_t)max(m.x, m.y) << 16;
}
MOE_DEV uint32_t magnitude4(const u32x4& v) {  // 4 FP32 values
  return max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
}
MOE_DEV uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, kWave));
  return v;
}

// A row is read once and its codes are read next: the row's lines need not stay in the L2 (8192 rows of 7168 values with
// the L2 cold 36 -> 34 us on one card, dispatch of 16K tokens 20 -> 18.6 us; codes stored past the L2 cost the GEMM more).
MOE_DEV u32x4 load_once(const u32x4* p) {
  const i32x4_t v = __builtin_nontemporal_load((const i32x4_t*)p);
  return u32x4{(uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3]};
}

// One wave: the row's scale, its codes handed out vector by vector. NV > 0: the row stays in
// registers (nvec <= 64 NV); NV = 0: it is read twice.
template <int NV, class Out>
MOE_DEV RowScale quantize_row(const u32x4* src, int64_t nvec, int lane, Out&& out) {
  uint32_t m = 0;
  if constexpr (NV > 0) {
    u32x4 v[NV];
#pragma unroll
    for (int b = 0; b < NV; ++b) {
      const int64_t i = b * 64 + lane;
      v[b] = i < nvec ? load_once(src + i) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int b = 0; b < NV; ++b) m = max(m, magnitude8(v[b]));
    const RowScale r = row_scale(wave_max_u32(m));
#pragma unroll
    for (int b = 0; b < NV; ++b) {
      const int64_t i = b * 64 + lane;
      if (i < nvec) out(i, codes8(v[b], r.inv));
    }
    return r;
  } else {
    for (int64_t i = lane; i < nvec; i += 64) m = max(m, magnitude8(src[i]));
    const RowScale r = row_scale(wave_max_u32(m));
    for (int64_t i = lane; i < nvec; i += 64) out(i, codes8(src[i], r.inv));
    return r;
  }
}

template <int NV>
__global__ __launch_bounds__(256) void quantize_rows_i8_kernel(const u32x4* __restrict__ src, uint2* __restrict__ codes,
                                                               float* __restrict__ scale, int64_t rows, int64_t nvec) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * kI8RowsPerBlock + (threadIdx.x >> 6);
  if (r >= rows) return;
  uint2* dst = codes + r * nvec;
  const RowScale q = quantize_row<NV>(src + r * nvec, nvec, lane, [&](int64_t i, uint2 c) { dst[i] = c; });
  if (lane == 0) scale[r] = q.scale;
}

// Dispatch: x[t] quantised once and stored to every local slot's row. Many tokens: one wave per token,
// a token without a local slot is not read (19 us at 16K tokens of 2048 with 16 of 128 experts local; a
// block per token 22 us).
template <int NV>
__global__ __launch_bounds__(256) void dispatch_i8_kernel(const u32x4* __restrict__ x, const int32_t* __restrict__ row_of,
                                                          uint2* __restrict__ xd, float* __restrict__ xd_scale, int64_t t0,
                                                          int64_t t1, int K, int64_t nvec) {
  const int lane = threadIdx.x & 63;
  const int64_t t = t0 + (int64_t)blockIdx.x * kI8RowsPerBlock + (threadIdx.x >> 6);
  if (t >= t1) return;
  const int32_t myrow = lane < K ? row_of[t * K + lane] : -1;
  if (__ballot(myrow >= 0) == 0) return;
  const RowScale q = quantize_row<NV>(x + t * nvec, nvec, lane, [&](int64_t i, uint2 c) {
    for (int j = 0; j < K; ++j) {
      const int32_t r = __builtin_amdgcn_readlane(myrow, j);
      if (r >= 0) xd[(int64_t)r * nvec + i] = c;
    }
  });
  if (myrow >= 0) xd_scale[myrow] = q.scale;
}

// Up to 2048 tokens are bound by latency (one token 4.5 -> 2.6 us, 1341 of 4096 values 10.9 -> 9.1 us, 8192 of 512 with
// few local 5.2 and 6.7 us): one block per token, whose values load beside
// its slots without a check; thread i holds vectors i, i + 256, ... (NV = 0: read twice).
constexpr int kDispThreads = 256;
template <int NV>
__global__ __launch_bounds__(kDispThreads) void dispatch_few_i8_kernel(const u32x4* __restrict__ x, const int32_t* __restrict__ row_of,
                                                                   uint2* __restrict__ xd, float* __restrict__ xd_scale,
                                                                   int64_t t0, int K, int64_t nvec) {
  __shared__ uint32_t part[kDispThreads / 64];
  const int lane = threadIdx.x & 63;
  const int64_t t = t0 + blockIdx.x;
  const int32_t myrow = lane < K ? row_of[t * K + lane] : -1;
  const u32x4* src = x + t * nvec;
  u32x4 v[NV > 0 ? NV : 1];
  uint32_t m = 0;
  if constexpr (NV > 0) {
#pragma unroll
    for (int b = 0; b < NV; ++b) {
      const int64_t i = threadIdx.x + b * kDispThreads;
      v[b] = i < nvec ? src[i] : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int b = 0; b < NV; ++b) m = max(m, magnitude8(v[b]));
  } else {
    for (int64_t i = threadIdx.x; i < nvec; i += kDispThreads) m = max(m, magnitude8(src[i]));
  }
  m = wave_max_u32(m);
  if (lane == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  m = part[0];
#pragma unroll
  for (int w = 1; w < kDispThreads / 64; ++w) m = max(m, part[w]);
  const RowScale q = row_scale(m);
  auto store = [&](int64_t i, uint2 c) {
    for (int j = 0; j < K; ++j) {
      const int32_t r = __builtin_amdgcn_readlane(myrow, j);
      if (r >= 0) xd[(int64_t)r * nvec + i] = c;
    }
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int b = 0; b < NV; ++b) {
      const int64_t i = threadIdx.x + b * kDispThreads;
      if (i < nvec) store(i, codes8(v[b], q.inv));
    }
  } else {
    for (int64_t i = threadIdx.x; i < nvec; i += kDispThreads) store(i, codes8(src[i], q.inv));
  }
  if (threadIdx.x < 64 && myrow >= 0) xd_scale[myrow] = q.scale;
}

// The FP32 rows of h of each chunk (the row count is on the device): 4 values a vector.
template <int NV>
__global__ __launch_bounds__(256) void quantize_h_i8_kernel(const u32x4* __restrict__ src, uint32_t* __restrict__ codes,
                                                            float* __restrict__ scale, const int32_t* __restrict__ offsets,
                                                            int El, int c0, int64_t P_c, int64_t nvec) {
  const int lane = threadIdx.x & 63;
  const int c = c0 + (int)blockIdx.y;
  const int64_t n = min((int64_t)offsets[(int64_t)c * (El + 1) + El], P_c);  // no row past the chunk, whatever the table holds
  for (int64_t r = (int64_t)blockIdx.x * kI8RowsPerBlock + (threadIdx.x >> 6); r < n;
       r += (int64_t)gridDim.x * kI8RowsPerBlock) {
    const int64_t row = (int64_t)c * P_c + r;
    const u32x4* s = src + row * nvec;
    uint32_t* dst = codes + row * nvec;
    uint32_t m = 0;
    auto code = [](const u32x4& v, float inv) {
      return codes4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w), inv);
    };
    RowScale q;
    if constexpr (NV > 0) {
      u32x4 v[NV];
#pragma unroll
      for (int b = 0; b < NV; ++b) {
        const int64_t i = b * 64 + lane;
        v[b] = i < nvec ? s[i] : u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int b = 0; b < NV; ++b) m = max(m, magnitude4(v[b]));
      q = row_scale(wave_max_u32(m));
#pragma unroll
      for (int b = 0; b < NV; ++b) {
        const int64_t i = b * 64 + lane;
        if (i < nvec) dst[i] = code(v[b], q.inv);
      }
    } else {
      for (int64_t i = lane; i < nvec; i += 64) m = max(m, magnitude4(s[i]));
      q = row_scale(wave_max_u32(m));
      for (int64_t i = lane; i < nvec; i += 64) dst[i] = code(s[i], q.inv);
    }
    if (lane == 0) scale[row] = q.scale;
  }
}

static inline dim3 row_grid(int64_t n) { return dim3((unsigned)((n + kI8RowsPerBlock - 1) / kI8RowsPerBlock)); }

// vectors per lane: the smallest of 1, 2, 4, 8, 16 that holds the row, 0 (two reads) above
#define MOE_I8_NV(nvec, ...)                                                  \
  do {                                                                        \
    if ((nvec) <= 64) { constexpr int NV = 1; __VA_ARGS__; }                  \
    else if ((nvec) <= 128) { constexpr int NV = 2; __VA_ARGS__; }            \
    else if ((nvec) <= 256) { constexpr int NV = 4; __VA_ARGS__; }            \
    else if ((nvec) <= 512) { constexpr int NV = 8; __VA_ARGS__; }            \
    else if ((nvec) <= 64 * kI8MaxVec) { constexpr int NV = 16; __VA_ARGS__; }\
    else { constexpr int NV = 0; __VA_ARGS__; }                               \
  } while (0)

hipError_t launch_quantize_rows_i8(const void* src, void* codes, float* scale, int64_t rows, int cols, hipStream_t s) {
  if (rows <= 0) return hipSuccess;
  const int64_t nvec = cols / 8;
  {
    MOE_TRACE("quantize_rows_i8", s);
    MOE_I8_NV(nvec, MOE_LAUNCH(quantize_rows_i8_kernel<NV>, row_grid(rows), dim3(256), 0, s, (const u32x4*)src,
                               (uint2*)codes, scale, rows, nvec));
  }
  return hipGetLastError();
}

hipError_t launch_dispatch_i8(const void* x, const int32_t* row_of, void* xd, float* xd_scale, int64_t t0, int64_t t1,
                              int K, int H, hipStream_t s) {
  if (t1 <= t0) return hipSuccess;
  const int64_t nvec = H / 8;
  {
    MOE_TRACE("dispatch_i8", s);
    if (t1 - t0 > 2048) {
      MOE_I8_NV(nvec, MOE_LAUNCH(dispatch_i8_kernel<NV>, row_grid(t1 - t0), dim3(256), 0, s, (const u32x4*)x, row_of,
                                 (uint2*)xd, xd_scale, t0, t1, K, nvec));
    } else {
      auto k = nvec <= kDispThreads       ? dispatch_few_i8_kernel<1>
               : nvec <= 2 * kDispThreads ? dispatch_few_i8_kernel<2>
               : nvec <= 4 * kDispThreads ? dispatch_few_i8_kernel<4>
                                          : dispatch_few_i8_kernel<0>;
      MOE_LAUNCH(k, dim3((unsigned)(t1 - t0)), dim3(kDispThreads), 0, s, (const u32x4*)x, row_of, (uint2*)xd, xd_scale, t0,
                 K, nvec);
    }
  }
  return hipGetLastError();
}

hipError_t launch_quantize_h_i8(const float* h, void* codes, float* scale, const int32_t* offsets, int El, int c0, int nc,
                                int64_t P_c, int cols, hipStream_t s) {
  if (nc <= 0 || El <= 0) return hipSuccess;
  const int64_t nvec = cols / 4;
  const unsigned gx = (unsigned)std::max<int64_t>(1, std::min<int64_t>((P_c + kI8RowsPerBlock - 1) / kI8RowsPerBlock, 4096));
  {
    MOE_TRACE("quantize_h_i8", s);
    MOE_I8_NV(nvec, MOE_LAUNCH(quantize_h_i8_kernel<NV>, dim3(gx, (unsigned)nc), dim3(256), 0, s, (const u32x4*)h,
                               (uint32_t*)codes, scale, offsets, El, c0, P_c, nvec));
  }
  return hipGetLastError();
}

}  // namespace moe
