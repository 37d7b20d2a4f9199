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
// (No pointer here is declared apart from others: outputs may be inputs.)
// I: the type of column indexes, int where a row's length allows (32-bit
// compares, and a row base in scalar registers with a 32-bit offset).
template <class T, int N, class I>
__device__ __forceinline__ void load_row(const T* row, I c, I cols, float fill, float (&v)[N]) {
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

template <class T, int N, class I>
__device__ __forceinline__ void store_row(T* row, I c, I cols, const float (&v)[N]) {
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

// store_row with nontemporal stores.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <class T, int N, class I>
__device__ __forceinline__ void stream_row(T* row, I c, I cols, const float (&v)[N]) {
  if (c + N <= cols) {
    T t[N];
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = from_f32<T>(v[e]);
    u32x4_any u;
    static_assert(sizeof(u) == sizeof(t), "a 16-byte vector");
    __builtin_memcpy(&u, t, sizeof(t));
    __builtin_nontemporal_store(u, reinterpret_cast<u32x4_any*>(row + c));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < cols) row[c + e] = from_f32<T>(v[e]);
  }
}

// load_row in two steps, for a load issued ahead of its use: the N values as
// they are stored (those beyond `cols` are `fill`), then as floats.
template <class T, int N>
struct RawRow {
  T t[N];
  template <class I>
  __device__ __forceinline__ void load(const T* row, I c, I cols, T fill = T{}) {
    if (c + N <= cols) {
      __builtin_memcpy(t, row + c, sizeof(t));
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) t[e] = c + e < cols ? row[c + e] : fill;
    }
  }
  __device__ __forceinline__ float operator[](int e) const { return to_f32(t[e]); }
};

// The low bytes of four integers as one word.
__device__ __forceinline__ uint32_t pack_bytes(int a, int b, int c, int d) {
  return __builtin_amdgcn_perm(b, a, 0x0C0C0400u) | __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
}

// N int8 codes at row[c ...], four to a word; those beyond `cols` are 0.
// (Kept as words, a code becomes a float in one instruction; as bytes, every
// one is moved on its own.)
template <int N>
struct CodeWords {
  uint32_t w[N / 4];
  template <class I>
  __device__ __forceinline__ void load(const int8_t* row, I c, I cols) {
    if (c + N <= cols) {
      __builtin_memcpy(w, row + c, N);
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + 4 * i + e < cols) w[i] |= (uint32_t)(uint8_t)row[c + 4 * i + e] << (8 * e);
      }
    }
  }
  __device__ __forceinline__ float operator[](int e) const {
    return (float)(int)(int8_t)(w[e / 4] >> (8 * (e % 4)));
  }
};

template <int N, class I>
__device__ __forceinline__ void store_codes(int8_t* row, I c, I cols, const int (&q)[N]) {
  if (c + N <= cols) {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      w[i] = pack_bytes(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
    __builtin_memcpy(row + c, w, N);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < cols) row[c + e] = (int8_t)q[e];
  }
}

// Reductions over aligned groups of lanes: the lanes at distance 1, 2, 4, 8
// are reached with DPP (a group that already holds one value may be mirrored
// instead), those at 16 and 32 with the row swaps of gfx950, which leave the
// two values of a pair in two registers.  All of it stays in the vector ALU;
// a butterfly through LDS (ds_bpermute) takes several times as long a step.
template <int STEP>
__device__ __forceinline__ uint32_t lane_partner(uint32_t v) {
  constexpr int ctrl = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;   // quad_perm, quad_perm,
  return __builtin_amdgcn_update_dpp(0, v, ctrl, 0xF, 0xF, true);                         // half mirror, mirror
}

struct Pair32 {
  uint32_t a, b;
};
template <int STEP>
__device__ __forceinline__ Pair32 lane_pair(uint32_t v) {
  if constexpr (STEP == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return Pair32{r[0], r[1]};
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return Pair32{r[0], r[1]};
  }
}

template <int STEP>
__device__ __forceinline__ double lane_add_f64(double v) {
  const uint64_t x = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)x, hi = (uint32_t)(x >> 32);
  if constexpr (STEP < 16) {
    return v + __builtin_bit_cast(double, (uint64_t)lane_partner<STEP>(hi) << 32 | lane_partner<STEP>(lo));
  } else {
    const Pair32 l = lane_pair<STEP>(lo), h = lane_pair<STEP>(hi);
    return __builtin_bit_cast(double, (uint64_t)h.a << 32 | l.a) + __builtin_bit_cast(double, (uint64_t)h.b << 32 | l.b);
  }
}

// Sum over the wavefront in binary64, the same value in every lane (both
// lanes of a pair add the same two values).
__device__ __forceinline__ double wave_sum_f64(double v) {
  v = lane_add_f64<1>(v);
  v = lane_add_f64<2>(v);
  v = lane_add_f64<4>(v);
  v = lane_add_f64<8>(v);
  v = lane_add_f64<16>(v);
  return lane_add_f64<32>(v);
}

// Maximum over aligned groups of LANES lanes (a power of two).
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max_u32(uint32_t v) {
  if constexpr (LANES > 1) v = max(v, lane_partner<1>(v));
  if constexpr (LANES > 2) v = max(v, lane_partner<2>(v));
  if constexpr (LANES > 4) v = max(v, lane_partner<4>(v));
  if constexpr (LANES > 8) v = max(v, lane_partner<8>(v));
  if constexpr (LANES > 16) {
    const Pair32 p = lane_pair<16>(v);
    v = max(p.a, p.b);
  }
  if constexpr (LANES > 32) {
    const Pair32 p = lane_pair<32>(v);
    v = max(p.a, p.b);
  }
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

// exp(x) 2^-k, with k in the low bits of t: x = k ln2 + r with k the nearest
// integer to x / ln2 (found by adding 1.5 * 2^23) and |r| <= ln2/2, ln2 in two
// parts of which the first has 9 trailing zeros, so that its product is exact;
// then 1 + r + r^2 q(r), q of degree 4 fitted to e^r with relative error
// 3.8e-9.  IEEE operations throughout; the result is off by less than
// 1.3 * 2^-24 relative.
__device__ __forceinline__ float exp_reduced(float x, uint32_t& t) {
  const float big = __builtin_fmaf(x, 1.44269504f, 12582912.0f);
  t = __float_as_uint(big);
  const float k = big - 12582912.0f;
  float r = __builtin_fmaf(k, -0.693145752f, x);
  r = __builtin_fmaf(k, -1.42860677e-6f, r);
  float p = 0.00138145988f;
  p = __builtin_fmaf(p, r, 0.00836871658f);
  p = __builtin_fmaf(p, r, 0.041668389f);
  p = __builtin_fmaf(p, r, 0.166665211f);
  p = __builtin_fmaf(p, r, 0.49999994f);
  p = __builtin_fmaf(p, r, 1.0f);
  return __builtin_fmaf(p, r, 1.0f);
}

// exp(x) for x up to 88: +0 from -104 down, NaN for a NaN (v_maximum3 keeps it).
__device__ __forceinline__ float exp_f32(float x) {
  uint32_t t;
  const float p = exp_reduced(__builtin_elementwise_maximum(x, -104.0f), t);
  return __builtin_ldexpf(p, (int)(t - 0x4B400000u));
}

// exp(x) for -87.4 < x <= 0 (a result below 2^-126 is not exact).
__device__ __forceinline__ float exp_small(float x) {
  uint32_t t;
  const float p = exp_reduced(x, t);
  return __uint_as_float(__float_as_uint(p) + (t << 23));
}

// 1 / a for 1 <= a <= 2: the quadratic whose error T3(2a-3)/99 is the least
// (1% relative), and two Newton steps; off by less than 1.2 * 2^-24 relative.
__device__ __forceinline__ float recip_1_2(float a) {
  float y = __builtin_fmaf(__builtin_fmaf(32.0f / 99.0f, a, -144.0f / 99.0f), a, 210.0f / 99.0f);
  y = __builtin_fmaf(y, __builtin_fmaf(-a, y, 1.0f), y);
  return __builtin_fmaf(y, __builtin_fmaf(-a, y, 1.0f), y);
}

}  // namespace i8g
