// i8g_row.h -- device helpers of the row operators (norm.hip, checkpoint.hip,
// logprob.hip): typed 16-byte loads and stores of any alignment, sums over a
// wavefront in binary64, and the exponential.
#pragma once
#include "i8g_device.h"

namespace i8g {

struct bf16_t { uint16_t bits; };
struct f16_t { _Float16 v; };

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16_t x) { return __uint_as_float((uint32_t)x.bits << 16); }
__device__ __forceinline__ float to_f32(f16_t x) { return (float)x.v; }

// Round to nearest-even (the hardware conversions; NaN stays NaN, values
// beyond the type's range become infinite).
template <class T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ bf16_t from_f32<bf16_t>(float x) {
  return bf16_t{__builtin_bit_cast(uint16_t, (__bf16)x)};
}
template <> __device__ __forceinline__ f16_t from_f32<f16_t>(float x) { return f16_t{(_Float16)x}; }

// Values of one 16-byte vector: 4 f32, 8 bf16 or f16.
template <class T> constexpr int kVec = 16 / (int)sizeof(T);

// N consecutive values at row[c ...] as floats; values at and beyond `cols`
// read as `fill` (nothing outside the row is touched).  A full vector is one
// load of any alignment (gfx950 code objects run with unaligned access on).
template <class T, int N>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int64_t c, int64_t cols, float fill,
                                         float (&v)[N]) {
  if (c + N <= cols) {
    T t[N];
    __builtin_memcpy(t, row + c, sizeof(t));
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = to_f32(t[e]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = c + e < cols ? to_f32(row[c + e]) : fill;
  }
}

template <class T, int N>
__device__ __forceinline__ void store_row(T* __restrict__ row, int64_t c, int64_t cols, const float (&v)[N]) {
  if (c + N <= cols) {
    T t[N];
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = from_f32<T>(v[e]);
    __builtin_memcpy(row + c, t, sizeof(t));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < cols) row[c + e] = from_f32<T>(v[e]);
  }
}

// N int8 codes at row[c ...]; those beyond `cols` are 0.
template <int N>
__device__ __forceinline__ void load_codes(const int8_t* __restrict__ row, int64_t c, int64_t cols,
                                           int (&q)[N]) {
  int8_t t[N];
  if (c + N <= cols) {
    __builtin_memcpy(t, row + c, N);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = c + e < cols ? row[c + e] : (int8_t)0;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) q[e] = t[e];
}

template <int N>
__device__ __forceinline__ void store_codes(int8_t* __restrict__ row, int64_t c, int64_t cols,
                                            const int (&q)[N]) {
  if (c + N <= cols) {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      w[i] = (uint32_t)(q[4 * i] & 0xFF) | (uint32_t)(q[4 * i + 1] & 0xFF) << 8 |
             (uint32_t)(q[4 * i + 2] & 0xFF) << 16 | (uint32_t)(q[4 * i + 3] & 0xFF) << 24;
    __builtin_memcpy(row + c, w, N);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < cols) row[c + e] = (int8_t)q[e];
  }
}

// A lane's value exchanged with the lane at the given distance inside its
// aligned group of 2 * distance lanes; the groups below it must already hold
// one value (a reduction's steps 1, 2, 4, ..., 32 in this order).
template <int STEP>
__device__ __forceinline__ uint32_t lane_partner(uint32_t v) {
  if constexpr (STEP == 1) return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);    // quad 1,0,3,2
  if constexpr (STEP == 2) return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);    // quad 2,3,0,1
  if constexpr (STEP == 4) return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);   // row_half_mirror
  if constexpr (STEP == 8) return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true);   // row_mirror
  if constexpr (STEP == 16 || STEP == 32) return __shfl_xor((int)v, STEP, 64);
}

template <int STEP>
__device__ __forceinline__ double lane_partner_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = lane_partner<STEP>((uint32_t)b), hi = lane_partner<STEP>((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the wavefront in binary64, the same value in every lane (each
// step adds a pair in either order, which gives the same bits).
__device__ __forceinline__ double wave_sum_f64(double v) {
  v += lane_partner_f64<1>(v);
  v += lane_partner_f64<2>(v);
  v += lane_partner_f64<4>(v);
  v += lane_partner_f64<8>(v);
  v += lane_partner_f64<16>(v);
  v += lane_partner_f64<32>(v);
  return v;
}

// Maximum over aligned groups of LANES lanes (a power of two).
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max_u32(uint32_t v) {
  if constexpr (LANES > 1) v = max(v, lane_partner<1>(v));
  if constexpr (LANES > 2) v = max(v, lane_partner<2>(v));
  if constexpr (LANES > 4) v = max(v, lane_partner<4>(v));
  if constexpr (LANES > 8) v = max(v, lane_partner<8>(v));
  if constexpr (LANES > 16) v = max(v, lane_partner<16>(v));
  if constexpr (LANES > 32) v = max(v, lane_partner<32>(v));
  return v;
}

// |x| as an integer that orders like it; NaN and infinity are the largest.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;

// The scale of a line from the largest abs_bits of its values: the rule of
// quantize_rows, and NaN for a line that holds an infinity or a NaN.
__device__ __forceinline__ float scale_of_bits(uint32_t a) {
  return a < kInfBits ? scale_of_absmax(__uint_as_float(a)) : __uint_as_float(0x7FC00000u);
}

// exp(x), for x up to about 80; +0 below -104; in IEEE operations: x = k
// ln2 + r with |r| <= ln2/2 (ln2 in two parts, the fused steps exact enough
// that r is off by less than an ulp), the Taylor polynomial of degree 7 (its
// remainder is below 2^-28), scaled by 2^k.
__device__ __forceinline__ float exp_neg(float x) {
  x = x < -104.0f ? -104.0f : x;                          // (a NaN stays)
  const float k = __builtin_rintf(x * 1.44269504f);
  float r = __builtin_fmaf(k, -0.693145752f, x);          // 0x3F317200: 9 trailing zeros, k * ln2hi is exact
  r = __builtin_fmaf(k, -1.42860677e-6f, r);
  float p = 1.98412698e-4f;
  p = __builtin_fmaf(p, r, 1.38888889e-3f);
  p = __builtin_fmaf(p, r, 8.33333333e-3f);
  p = __builtin_fmaf(p, r, 4.16666667e-2f);
  p = __builtin_fmaf(p, r, 1.66666667e-1f);
  p = __builtin_fmaf(p, r, 0.5f);
  p = __builtin_fmaf(p, r, 1.0f);
  p = __builtin_fmaf(p, r, 1.0f);
  return __builtin_ldexpf(p, (int)k);
}

}  // namespace i8g
