// norm.hip -- layer norm: forward (to values or to the int8 codes of the
// next GEMM's A operand) and backward with the reduction of the weight's and
// the bias's gradient.
//
// Forward, for a row x of n values (the sums in binary64, everything else in
// separately rounded binary32 steps):
//   mean = RN(sum x / n)      rstd = RN(1 / sqrt(sum (x-m)^2 / n + eps))
//   y_j  = RN(RN(RN(RN(x_j - mean) * rstd) * gamma_j) + beta_j)
// Backward, for the gradient dy of y:
//   xh = RN(RN(x - mean) * rstd)      w  = RN(dy * gamma)
//   c1 = RN(sum w / n)                c2 = RN(sum w*xh / n)
//   dx = RN(rstd * RN(RN(w - c1) - RN(xh * c2)))
//   dgamma_j = RN(sum over rows of dy*xh)     dbeta_j = RN(sum over rows of dy)
// A product of two binary32 values is exact in binary64, and a binary64 sum of
// k of them one after another is off by at most k 2^-53 of its terms'
// magnitude, k being the values of a lane or the rows of a workgroup: less
// than 2^-40 up to 2^20 rows, 2^-29 for 2^31.  So the rounded sums do not
// depend on the order of addition except next to a rounding border; the order
// is fixed by the sizes all the same (no atomics), so two runs give the same
// bytes.
//
// Both directions are bound by memory: a value is read once and written once,
// a row staying in registers in between.  A row of up to 1024 values is held by
// one wave, 16 values a lane; a longer one by 2 to 16 waves of one workgroup;
// rows beyond 16384 values are read again instead of held.  The backward pass
// reads rows beyond 8192 values twice: the sums over the rows do not fit the
// registers beside them and are a pass of their own.
//
// 8192 x 768 f32, which the 256 MB cache holds (a copy there moves 6.9 TB/s):
// forward 10.0 us (50 MB, 5.0 TB/s), into codes 10.6 us (31 MB), backward 15.5 us
// (75 MB, 4.9 TB/s) and 3.9 us for the columns' sums.  About 2 us of each are
// the launch and the first load; in codes the row's second reduction, which
// waits for the first, and the quantizing are most of the rest.
#include <type_traits>

#include "i8g_launch.h"
#include "i8g_row.h"

namespace i8g {
namespace {

constexpr int kHeldMax = 16384;      // longest row held in registers: 16 waves of 64 lanes x 16 values

// 1 / sqrt(a) in binary64: the hardware's estimate (relative error below
// 2^-20) and one third-order step.
__device__ __forceinline__ double rsqrt_f64(double a) {
  if (a == 0.0) return __builtin_huge_val();
  const double y = __builtin_amdgcn_rsq(a);
  const double e = __builtin_fma(-a * y, y, 1.0);
  return __builtin_fma(y * e, __builtin_fma(0.375, e, 0.5), y);
}

// Row sums of two binary64 values over the W waves (consecutive ones of the
// workgroup) that share a row; the result is in every lane.  `red` has two
// halves used in turn, so one barrier per call is enough: a wave can reach the
// call after the next one only when every wave has read this one's half.
template <int W>
__device__ __forceinline__ void row_sum2(double& a, double& b, double (*red)[2 * W], int& turn) {
  a = wave_sum_f64(a);
  b = wave_sum_f64(b);
  if constexpr (W > 1) {
    double* half = red[turn];
    turn ^= 1;
    const int wave = (threadIdx.x >> 6) % W;
    if ((threadIdx.x & 63) == 0) {
      half[wave] = a;
      half[W + wave] = b;
    }
    __syncthreads();
    a = 0.0;
    b = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      a += half[w];
      b += half[W + w];
    }
  }
}

template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t (*red)[W], int& turn) {
  v = lanes_max_u32<64>(v);
  if constexpr (W > 1) {
    uint32_t* half = red[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) half[(threadIdx.x >> 6) % W] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) v = max(v, half[w]);
  }
  return v;
}

struct RowStats {
  float mean, rstd;
};

// s1 = sum (x - x0), s2 = sum (x - x0)^2 with the row's first value x0 as the
// pivot: it lies within sqrt(n) standard deviations of the mean, so
// s2 - s1^2/n loses at most a factor n of binary64's 2^-53.
__device__ __forceinline__ RowStats stats_of(double x0, double s1, double s2, double inv_n, double eps) {
  const double d = s1 * inv_n;
  double var = s2 * inv_n - d * d;
  var = var < 0.0 ? 0.0 : var;            // (a NaN stays)
  return RowStats{(float)(x0 + d), (float)rsqrt_f64(var + eps)};
}

// Rows held in registers; the workgroups walk the rows with a fixed stride,
// the next row's values on their way while one is worked on, gamma and beta
// held throughout.
template <class T, int N, int NV, int W, bool QUANT>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W) ln_fwd_kernel(LnFwdArgs a) {
  __shared__ double red[2][2 * W];
  __shared__ uint32_t redm[2][W];
  int turn = 0, turnm = 0;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = (int)a.cols;
  const int64_t step = W == 1 ? (int64_t)gridDim.x * 4 : gridDim.x;
  const int c0 = (W == 1 ? 0 : wave * 64 * N * NV) + lane * N;
  const T* X = static_cast<const T*>(a.X);
  int64_t r = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  struct Row {
    RawRow<T, N> v[NV];
    T first;
  } cur;
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    const T* xr = X + row * a.ldx;
    cur.first = xr[0];
#pragma unroll
    for (int i = 0; i < NV; ++i) cur.v[i].load(xr, c0 + i * 64 * N, cols, cur.first);
  };
  if (r < a.rows) fetch(r);
  float g[NV][N], b[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * 64 * N;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      g[i][e] = c + e < cols ? 1.0f : 0.0f;             // behind the row's end y is 0
      b[i][e] = 0.0f;
    }
    if (a.gamma) load_row<float>(a.gamma, c, cols, 0.0f, g[i]);
    if (a.beta) load_row<float>(a.beta, c, cols, 0.0f, b[i]);
  }
  for (; r < a.rows; r += step) {
    float v[NV][N];
    const double x0 = to_f32(cur.first);
    double s1 = 0.0, s2 = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[i][e] = cur.v[i][e];
        const double d = (double)v[i][e] - x0;            // 0 behind the row's end
        s1 += d;
        s2 = __builtin_fma(d, d, s2);
      }
    }
    if (r + step < a.rows) fetch(r + step);
    row_sum2<W>(s1, s2, red, turn);
    const RowStats st = stats_of(x0, s1, s2, a.inv_n, a.eps);
    if ((W == 1 || wave == 0) && lane == 0) {
      if (a.mean) a.mean[r] = st.mean;
      if (a.rstd) a.rstd[r] = st.rstd;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * 64 * N;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float xh = mul_rn(add_rn(v[i][e], -st.mean), st.rstd);
        v[i][e] = add_rn(mul_rn(xh, g[i][e]), b[i][e]);
        if constexpr (QUANT) m = max(m, abs_bits(v[i][e]));
      }
      if (!QUANT) store_row<T>(static_cast<T*>(a.Y) + r * a.ldy, c, cols, v[i]);
    }
    if constexpr (QUANT) {
      m = row_max<W>(m, redm, turnm);
      const float s = scale_of_bits(m);
      const bool fine = m < kInfBits;
      const float inv = recip_rn(s);
      if ((W == 1 || wave == 0) && lane == 0) a.scale[r] = s;
      int8_t* qr = static_cast<int8_t*>(a.Y) + r * a.ldy;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        int q[N];
#pragma unroll
        for (int e = 0; e < N; ++e) q[e] = fine ? quantize1(v[i][e], inv) : 0;
        store_codes(qr, c0 + i * 64 * N, cols, q);
      }
    }
  }
}

// Rows that no workgroup holds: a workgroup of 16 waves per row, which reads
// the row again (from cache) for each step.
template <class T, bool QUANT>
__global__ void __launch_bounds__(1024) ln_fwd_long_kernel(LnFwdArgs a) {
  constexpr int N = kVec<T>;
  constexpr int64_t STEP = 1024 * N;
  __shared__ double red[2][32];
  __shared__ uint32_t redm[2][16];
  int turn = 0, turnm = 0;
  const int64_t c0 = (int64_t)threadIdx.x * N;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* xr = static_cast<const T*>(a.X) + r * a.ldx;
    const float x0f = to_f32(xr[0]);
    const double x0 = x0f;
    double s1 = 0.0, s2 = 0.0;
    for (int64_t c = c0; c < a.cols; c += STEP) {
      float v[N];
      load_row<T>(xr, c, a.cols, x0f, v);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const double d = (double)v[e] - x0;
        s1 += d;
        s2 = __builtin_fma(d, d, s2);
      }
    }
    row_sum2<16>(s1, s2, red, turn);
    const RowStats st = stats_of(x0, s1, s2, a.inv_n, a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = st.mean;
      if (a.rstd) a.rstd[r] = st.rstd;
    }
    auto values = [&](int64_t c, float (&v)[N]) __attribute__((always_inline)) {
      float g[N], b[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        g[e] = 1.0f;
        b[e] = 0.0f;
      }
      load_row<T>(xr, c, a.cols, x0f, v);
      if (a.gamma) load_row<float>(a.gamma, c, a.cols, 0.0f, g);
      if (a.beta) load_row<float>(a.beta, c, a.cols, 0.0f, b);
#pragma unroll
      for (int e = 0; e < N; ++e)
        v[e] = add_rn(mul_rn(mul_rn(add_rn(v[e], -st.mean), st.rstd), g[e]), b[e]);
    };
    uint32_t m = 0;
    if constexpr (QUANT) {
      for (int64_t c = c0; c < a.cols; c += STEP) {
        float v[N];
        values(c, v);
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (c + e < a.cols) m = max(m, abs_bits(v[e]));
      }
      m = row_max<16>(m, redm, turnm);
      if (threadIdx.x == 0) a.scale[r] = scale_of_bits(m);
    }
    const bool fine = m < kInfBits;
    const float inv = QUANT ? recip_rn(scale_of_bits(m)) : 0.0f;
    for (int64_t c = c0; c < a.cols; c += STEP) {
      float v[N];
      values(c, v);
      if constexpr (QUANT) {
        int q[N];
#pragma unroll
        for (int e = 0; e < N; ++e) q[e] = fine ? quantize1(v[e], inv) : 0;
        store_codes(static_cast<int8_t*>(a.Y) + r * a.ldy, c, a.cols, q);
      } else {
        store_row<T>(static_cast<T*>(a.Y) + r * a.ldy, c, a.cols, v);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  The input's values come from X, or are RN(q*s) of its 8-bit
// checkpoint (CK).
// ---------------------------------------------------------------------------
// N of them as they are stored.
template <class T, bool CK, int N>
struct Input : RawRow<T, N> {
  template <class I>
  __device__ __forceinline__ void load(const LnBwdArgs& a, int64_t r, I c) {
    RawRow<T, N>::load(static_cast<const T*>(a.X) + r * a.ldx, c, (I)a.cols);
  }
};
template <class T, int N>
struct Input<T, true, N> {
  CodeWords<N> q;
  float s;
  template <class I>
  __device__ __forceinline__ void load(const LnBwdArgs& a, int64_t r, I c) {
    q.load(static_cast<const int8_t*>(a.X) + r * a.ldx, c, (I)a.cols);
    s = c < (I)a.cols ? a.scale[r * a.lds + (c >> a.gshift)] : 0.0f;
  }
  __device__ __forceinline__ float operator[](int e) const { return mul_rn(q[e], s); }
};

__device__ __forceinline__ float bwd_xhat(float x, float mean, float rstd) { return mul_rn(add_rn(x, -mean), rstd); }
__device__ __forceinline__ float bwd_dx(float w, float xh, float rstd, float c1, float c2) {
  return mul_rn(rstd, add_rn(add_rn(w, -c1), -mul_rn(xh, c2)));
}

// Rows held in registers, by workgroups of 8 waves that hold 8/W rows at a
// time (16 waves and one row for W = 16) and walk the rows with a fixed
// stride, the next row's values on their way while one is worked on.  With
// PARTS each lane adds its columns' terms of dgamma and dbeta in binary64,
// and the workgroup leaves one partial sum per column in
// parts[block][2][held] for ln_bwd_cols_kernel, in the order of the lanes
// (column_of), which makes whole cache lines of them.
template <class T, bool CK, int N, int NV, int W, bool PARTS>
__global__ void __launch_bounds__(W == 16 ? 1024 : 512) ln_bwd_kernel(LnBwdArgs a) {
  constexpr int S = W == 16 ? 1 : 8 / W;
  __shared__ double red[S][2][2 * W];
  __shared__ double part[PARTS && S > 1 ? S : 1][PARTS && S > 1 ? NV * N * W * 64 : 1];
  int turn = 0;
  const int lane = threadIdx.x & 63, cols = (int)a.cols;
  const int slot = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) / W);
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % W);
  const int c0 = wave * 64 * N * NV + lane * N;
  float g[NV][N];
  double ag[PARTS ? NV : 1][N], ab[PARTS ? NV : 1][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      g[i][e] = 1.0f;
      if constexpr (PARTS) ag[i][e] = ab[i][e] = 0.0;
    }
    if (a.gamma) load_row<float>(a.gamma, c0 + i * 64 * N, cols, 0.0f, g[i]);
  }
  struct Row {
    Input<T, CK, N> x[NV];
    RawRow<T, N> dy[NV];
    float mean, rstd;
  } cur;
  auto fetch = [&](Row& w, int64_t r) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      w.x[i].load(a, r, c0 + i * 64 * N);
      w.dy[i].load(static_cast<const T*>(a.dY) + r * a.lddy, c0 + i * 64 * N, cols);
    }
    w.mean = a.mean[r];
    w.rstd = a.rstd[r];
  };
  const int64_t step = (int64_t)gridDim.x * S;
  int64_t first = (int64_t)blockIdx.x * S;               // the row of slot 0: the same for the workgroup
  if (first + slot < a.rows) fetch(cur, first + slot);
  for (; first < a.rows; first += step) {
    const int64_t r = first + slot;
    const bool live = r < a.rows;
    float x[NV][N], w[NV][N];
    double s1 = 0.0, s2 = 0.0;
    const float rstd = cur.rstd;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float dy = cur.dy[i][e], xh = bwd_xhat(cur.x[i][e], cur.mean, rstd);
          if constexpr (PARTS) {
            ag[i][e] = __builtin_fma((double)dy, (double)xh, ag[i][e]);   // (an exact product)
            ab[i][e] += (double)dy;
          }
          x[i][e] = xh;
          w[i][e] = mul_rn(dy, g[i][e]);
          s1 += (double)w[i][e];                          // (0 behind the row's end)
          // Behind the row's end dy and w are 0, but RN(0 - mean) * rstd may be infinite where no value of the row
          // has such an xh (equal ones, far out), and 0 times that is a NaN.  (Up to 2.5% of the pass; xh
          // itself set to 0 takes up to 5%, vectors that end and those that do not told apart 10%.)
          const bool inside = c0 + i * 64 * N + e < cols;
          s2 = __builtin_fma((double)w[i][e], (double)(inside ? xh : 0.0f), s2);
        }
      if (r + step < a.rows) fetch(cur, r + step);
    }
    if (a.dX) {                                           // (the same for the whole grid)
      row_sum2<W>(s1, s2, red[slot], turn);
      if (live) {
        const float c1 = (float)(s1 * a.inv_n), c2 = (float)(s2 * a.inv_n);
        T* dxr = static_cast<T*>(a.dX) + r * a.lddx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int e = 0; e < N; ++e) w[i][e] = bwd_dx(w[i][e], x[i][e], rstd, c1, c2);
          store_row<T>(dxr, c0 + i * 64 * N, cols, w[i]);
        }
      }
    }
  }
  if constexpr (PARTS) {
    constexpr int HELD = W * NV * N * 64;
    double* out = a.parts + (int64_t)blockIdx.x * 2 * HELD;
    if constexpr (S > 1) {
      // the slots' sums through LDS, added in the order of the slots; a column
      // per thread, first of dgamma, then of dbeta
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < N; ++e) part[slot][((wave * NV + i) * N + e) * 64 + lane] = k ? ab[i][e] : ag[i][e];
        __syncthreads();
        for (int j = threadIdx.x; j < HELD; j += 512) {
          double s = part[0][j];
#pragma unroll
          for (int q = 1; q < S; ++q) s += part[q][j];
          out[k * HELD + j] = s;
        }
        __syncthreads();
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int j = ((wave * NV + i) * N + e) * 64 + lane;
          out[j] = ag[i][e];
          out[HELD + j] = ab[i][e];
        }
    }
  }
}

// dx of rows that no workgroup holds.
template <class T, bool CK>
__global__ void __launch_bounds__(1024) ln_bwd_long_kernel(LnBwdArgs a) {
  constexpr int N = kVec<T>;
  constexpr int64_t STEP = 1024 * N;
  __shared__ double red[2][32];
  int turn = 0;
  const int64_t c0 = (int64_t)threadIdx.x * N;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* dyr = static_cast<const T*>(a.dY) + r * a.lddy;
    const float mean = a.mean[r], rstd = a.rstd[r];
    auto terms = [&](int64_t c, float (&x)[N], float (&w)[N]) __attribute__((always_inline)) {
      float g[N];
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] = 1.0f;
      Input<T, CK, N> in;
      in.load(a, r, c);
      load_row<T>(dyr, c, a.cols, 0.0f, w);
      if (a.gamma) load_row<float>(a.gamma, c, a.cols, 0.0f, g);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        x[e] = bwd_xhat(in[e], mean, rstd);
        w[e] = mul_rn(w[e], g[e]);
      }
    };
    double s1 = 0.0, s2 = 0.0;
    for (int64_t c = c0; c < a.cols; c += STEP) {
      float x[N], w[N];
      terms(c, x, w);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (c + e < a.cols) {
          s1 += (double)w[e];
          s2 = __builtin_fma((double)w[e], (double)x[e], s2);
        }
    }
    row_sum2<16>(s1, s2, red, turn);
    const float c1 = (float)(s1 * a.inv_n), c2 = (float)(s2 * a.inv_n);
    for (int64_t c = c0; c < a.cols; c += STEP) {
      float x[N], w[N];
      terms(c, x, w);
#pragma unroll
      for (int e = 0; e < N; ++e) w[e] = bwd_dx(w[e], x[e], rstd, c1, c2);
      store_row<T>(static_cast<T*>(a.dX) + r * a.lddx, c, a.cols, w);
    }
  }
}

// Partial sums of dgamma and dbeta for the same rows: a thread per vector of
// columns, blockIdx.y over the row ranges.
template <class T, bool CK>
__global__ void __launch_bounds__(64) ln_bwd_long_parts_kernel(LnBwdArgs a) {
  constexpr int N = kVec<T>;
  const int64_t c = ((int64_t)blockIdx.x * 64 + threadIdx.x) * N;
  if (c >= a.cols) return;
  double ag[N], ab[N];
#pragma unroll
  for (int e = 0; e < N; ++e) ag[e] = ab[e] = 0.0;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    Input<T, CK, N> x;
    float dy[N];
    x.load(a, r, c);
    load_row<T>(static_cast<const T*>(a.dY) + r * a.lddy, c, a.cols, 0.0f, dy);
    const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      ag[e] = __builtin_fma((double)dy[e], (double)bwd_xhat(x[e], mean, rstd), ag[e]);
      ab[e] += (double)dy[e];
    }
  }
  double* out = a.parts + (int64_t)blockIdx.y * 2 * a.cols;
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (c + e < a.cols) {
      out[c + e] = ag[e];
      out[a.cols + c + e] = ab[e];
    }
}

// The column of the j-th partial sum, lanes holding vectors of n values
// (n = 1: the sums are in the order of the columns).
__device__ __forceinline__ int64_t column_of(int64_t j, int n) {
  if (n == 1) return j;
  const int i = (int)j;                                   // (rows held by lanes are short)
  return n == 4 ? i / 256 * 256 + i % 64 * 4 + i / 64 % 4 : i / 512 * 512 + i % 64 * 8 + i / 64 % 8;
}

// 16 of the `held` partial sums (of dgamma, or with blockIdx.y of dbeta): a
// thread adds every 16th of one column (16 of them are one cache line of a
// partial), then the 16 threads of a column join.
__global__ void __launch_bounds__(256) ln_bwd_cols_kernel(const double* __restrict__ parts, int n_parts, int64_t held,
                                                          int order, int64_t cols, float* __restrict__ dgamma,
                                                          float* __restrict__ dbeta) {
  __shared__ double red[16][17];
  const int col = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int64_t j = (int64_t)blockIdx.x * 16 + col, c = column_of(j, order);
  float* const out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  double s = 0.0;
  if (c < cols) {
    const double* p = parts + blockIdx.y * held + j;
#pragma unroll 8
    for (int i = slice; i < n_parts; i += 16) s += p[(int64_t)i * 2 * held];
  }
  red[slice][col] = s;
  __syncthreads();
  if (slice == 0 && c < cols) {
#pragma unroll
    for (int w = 1; w < 16; ++w) s += red[w][col];
    out[c] = (float)s;
  }
}

// How a row is held: n values a vector, nv vectors a lane (16 values at most),
// in `waves` waves; the fewest that hold it.  Vectors are 16 bytes, but 8 in
// the 2-byte types for a row of one wave that whole vectors of 8 values would
// fill to less.  8192 x 768 bf16: into codes and restored 16.2 us with 4
// values a vector and 18.5 with 8, backward 14.3 and 18.1; 8192 x 1024, which
// both fill: 8.2 us with 8 and 10.9 with 4.  Longer rows take 3 vectors of 4
// where those hold them: 8192 x 1280 bf16 13.2 us and backward 23.7 (14.5 and
// 31.9 with 16 values a lane), 8192 x 6144 bf16 39.0 and 80.4 (46.0 and 80.2).
struct RowShape {
  int waves, n, nv;   // waves == 0: too long to hold
};
RowShape row_shape(int64_t cols, int vec) {
  if (cols > kHeldMax) return RowShape{0, vec, 0};
  const int64_t quarters = (cols + 255) / 256;           // of 64 lanes x 16 values
  if (quarters <= 4) {
    const int n = vec == 8 && quarters % 2 == 0 ? 8 : 4;
    return RowShape{1, n, (int)quarters * 4 / n};
  }
  int w = 2;
  while (w * 1024 < cols) w *= 2;
  const int n = cols <= w * 768 ? 4 : vec;
  return RowShape{w, n, cols <= w * 768 ? 3 : 16 / vec};
}

// Workgroups of a kernel whose workgroups walk the rows.
unsigned int row_grid(int64_t rows, int per_group, int64_t most) {
  const int64_t g = (rows + per_group - 1) / per_group;
  return (unsigned int)(g < most ? g : most);
}

// Calls f with the shape's N, NV and W as compile-time constants; V is the
// type's whole vector.  (A whole vector of 8 takes 1 or 2, a vector of 4 up to
// 4 in f32, and 1 or 3 where it is half of a whole one.)
template <int I>
using Int = std::integral_constant<int, I>;
template <int V, class F>
void with_shape(const RowShape& s, F f) {
  constexpr int M = 16 / V;
  switch (s.waves) {
    case 1:
      if constexpr (V == 8) {
        if (s.n == 8 && s.nv == 1) return f(Int<8>{}, Int<1>{}, Int<1>{});
        if (s.n == 8) return f(Int<8>{}, Int<2>{}, Int<1>{});
        if (s.nv == 1) return f(Int<4>{}, Int<1>{}, Int<1>{});
        return f(Int<4>{}, Int<3>{}, Int<1>{});
      } else {
        if (s.nv == 1) return f(Int<4>{}, Int<1>{}, Int<1>{});
        if (s.nv == 2) return f(Int<4>{}, Int<2>{}, Int<1>{});
        if (s.nv == 3) return f(Int<4>{}, Int<3>{}, Int<1>{});
        return f(Int<4>{}, Int<4>{}, Int<1>{});
      }
    case 2: return s.nv == 3 ? f(Int<4>{}, Int<3>{}, Int<2>{}) : f(Int<V>{}, Int<M>{}, Int<2>{});
    case 4: return s.nv == 3 ? f(Int<4>{}, Int<3>{}, Int<4>{}) : f(Int<V>{}, Int<M>{}, Int<4>{});
    case 8: return s.nv == 3 ? f(Int<4>{}, Int<3>{}, Int<8>{}) : f(Int<V>{}, Int<M>{}, Int<8>{});
    default: return s.nv == 3 ? f(Int<4>{}, Int<3>{}, Int<16>{}) : f(Int<V>{}, Int<M>{}, Int<16>{});
  }
}

template <class T, bool QUANT>
hipError_t ln_fwd(const LnFwdArgs& a, hipStream_t stream) {
  const RowShape s = row_shape(a.cols, kVec<T>);
  if (s.waves == 0) {
    const unsigned int grid = row_grid(a.rows, 1, int64_t(1) << 20);
    hipLaunchKernelGGL((ln_fwd_long_kernel<T, QUANT>), dim3(grid), dim3(1024), 0, stream, a);
  } else {
    with_shape<kVec<T>>(s, [&](auto n, auto nv, auto w) {
      constexpr int W = decltype(w)::value;
      const unsigned int grid = row_grid(a.rows, W == 1 ? 4 : 1, W == 1 ? 1024 : 4096 / W);
      hipLaunchKernelGGL((ln_fwd_kernel<T, decltype(n)::value, decltype(nv)::value, W, QUANT>), dim3(grid),
                         dim3(W == 1 ? 256 : 64 * W), 0, stream, a);
    });
  }
  return hipGetLastError();
}

template <class T, bool CK>
hipError_t ln_bwd(const LnBwdArgs& a, float* dgamma, float* dbeta, hipStream_t stream) {
  constexpr int V = kVec<T>;
  const int groups = ln_bwd_groups(a.rows, a.cols);
  const RowShape s = row_shape(a.cols, V);
  // Rows of 16 waves leave no registers for the sums over the rows, and
  // longer ones are not held: the sums are a pass of their own, before dX,
  // which may be dY's memory.
  const bool apart = s.waves == 0 || s.waves == 16;
  if (a.parts && apart)
    hipLaunchKernelGGL((ln_bwd_long_parts_kernel<T, CK>), dim3((unsigned int)((a.cols + 64 * V - 1) / (64 * V)), groups),
                       dim3(64), 0, stream, a);
  if (s.waves == 0) {
    if (a.dX && a.rows > 0)
      hipLaunchKernelGGL((ln_bwd_long_kernel<T, CK>), dim3(row_grid(a.rows, 1, int64_t(1) << 20)), dim3(1024), 0,
                         stream, a);
  } else {
    with_shape<V>(s, [&](auto n, auto nv, auto w) {
      constexpr int N = decltype(n)::value, NV = decltype(nv)::value, W = decltype(w)::value;
      if constexpr (W == 16) {
        if (a.dX && a.rows > 0)
          hipLaunchKernelGGL((ln_bwd_kernel<T, CK, N, NV, 16, false>), dim3(row_grid(a.rows, 1, 256)), dim3(1024), 0,
                             stream, a);
      } else if (a.parts) {
        hipLaunchKernelGGL((ln_bwd_kernel<T, CK, N, NV, W, true>), dim3(groups), dim3(512), 0, stream, a);
      } else {
        hipLaunchKernelGGL((ln_bwd_kernel<T, CK, N, NV, W, false>), dim3(row_grid(a.rows, 8 / W, 512)), dim3(512), 0,
                           stream, a);
      }
    });
  }
  if (a.parts) {
    const int64_t held = apart ? a.cols : (int64_t)s.waves * 64 * s.n * s.nv;
    const int order = apart ? 1 : s.n;
    // a launch holds fewer than 2^32 threads, 16 a column; a slab starts where
    // the columns are in order (only long rows take more than one)
    const int64_t slab = int64_t(1) << 27;
    for (int64_t j = 0; j < held; j += slab) {
      const int64_t n = held - j < slab ? held - j : slab;
      const int64_t cols = a.cols - j < slab ? a.cols - j : slab;
      hipLaunchKernelGGL(ln_bwd_cols_kernel, dim3((unsigned int)((n + 15) / 16), 2), dim3(256), 0, stream, a.parts + j,
                         groups, held, order, cols, dgamma ? dgamma + j : dgamma, dbeta ? dbeta + j : dbeta);
    }
  }
  return hipGetLastError();
}

}  // namespace

// Row ranges of the sums over the rows: one for each workgroup that walks the
// rows.  Where the sums are a pass of their own fewer do, since each leaves two
// binary64 values a column: 512 x 12288 bf16 35.7 us with 64, 40.4 with 128
// and 56.9 with 256; 2048 x 16384 107, 98 and 119; 8192 x 12288 320, 252 and 248.
int ln_bwd_groups(int64_t rows, int64_t cols) {
  if (cols > 8192) {
    const int64_t g = rows / 16 < 64 ? 64 : rows / 16 < 128 ? rows / 16 : 128;
    return (int)(rows < 1 ? 1 : rows < g ? rows : g);
  }
  const int per_group = cols <= 1024 ? 8 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1;
  const int64_t g = (rows + per_group - 1) / per_group;
  return (int)(g < 1 ? 1 : g < 256 ? g : 256);
}

// Partial sums of a workgroup of the backward pass, of one kind: the columns
// that its lanes hold (whole vectors of 8 values in 64 lanes, 1, 2, 4 or 8
// times 1024 of them in longer rows).
int64_t ln_bwd_held_max(int64_t cols) {
  if (cols <= 1024) return (cols + 511) / 512 * 512;
  for (int64_t held = 2048; held <= 8192; held *= 2)
    if (cols <= held) return held;
  return cols;
}

hipError_t launch_ln_fwd(const LnFwdArgs& a, int dtype, bool quant, hipStream_t stream) {
  switch (dtype) {
    case DT_F32: return quant ? ln_fwd<float, true>(a, stream) : ln_fwd<float, false>(a, stream);
    case DT_BF16: return quant ? ln_fwd<bf16_t, true>(a, stream) : ln_fwd<bf16_t, false>(a, stream);
    default: return quant ? ln_fwd<f16_t, true>(a, stream) : ln_fwd<f16_t, false>(a, stream);
  }
}

hipError_t launch_ln_bwd(const LnBwdArgs& a, int dtype, bool from_codes, float* dgamma, float* dbeta,
                         hipStream_t stream) {
  switch (dtype) {
    case DT_F32:
      return from_codes ? ln_bwd<float, true>(a, dgamma, dbeta, stream) : ln_bwd<float, false>(a, dgamma, dbeta, stream);
    case DT_BF16:
      return from_codes ? ln_bwd<bf16_t, true>(a, dgamma, dbeta, stream) : ln_bwd<bf16_t, false>(a, dgamma, dbeta, stream);
    default:
      return from_codes ? ln_bwd<f16_t, true>(a, dgamma, dbeta, stream) : ln_bwd<f16_t, false>(a, dgamma, dbeta, stream);
  }
}

}  // namespace i8g
