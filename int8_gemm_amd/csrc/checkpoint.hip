// checkpoint.hip -- activation checkpoints in 8 bits and their use in the
// backward pass.  A checkpoint is the quantize_rows rule applied to each
// group of 32 to 256 columns of a row: s = max(RN(a/127), RN(1e-8)),
// q = floor(RN(RN(x*RN(1/s)) + 0.5)), and stands for RN(q*s).  A group that
// holds an infinity or a NaN gets a NaN scale, so it restores as NaN.
//
// Storing reads a value and writes a byte; restoring, the activation's
// gradient and the column quantization of a checkpoint read that byte where
// they would have read a value.  All are bound by memory.
#include "i8g_launch.h"
#include "i8g_row.h"

namespace i8g {
namespace {

constexpr int kBlock = 256;

// The units of a matrix (N columns each, `per_row` of them in a row) are
// numbered row by row, a lane takes one, and so short and odd rows leave no
// lanes idle.  A launch covers fewer than 2^31 units (more rows take more
// launches), so the division by per_row is one multiplication: with
// 2^(l-1) < d <= 2^l and m = floor(2^(31+l) / d) + 1, n m / 2^(31+l) exceeds
// n / d by less than 1/d for n < 2^31, and its floor is exact.
struct Units {
  uint32_t per_row, mul, shift;
  __host__ explicit Units(uint32_t d) : per_row(d) {
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    shift = 31 + l;
    mul = (uint32_t)((uint64_t(1) << shift) / d + 1);
  }
  __device__ __forceinline__ uint32_t row(uint32_t n) const { return (uint32_t)((uint64_t)n * mul >> shift); }
};

// Units a row takes: whole groups of GROUP columns.
Units units_of(int64_t cols, int group, int n) { return Units((uint32_t)((cols + group - 1) / group * (group / n))); }

template <class T, int GROUP>
__global__ void __launch_bounds__(kBlock) checkpoint_store_kernel(const T* __restrict__ X, int64_t ldx, Checkpoint c,
                                                                  Units units) {
  constexpr int N = kVec<T>, LANES = GROUP / N;
  const uint32_t at = blockIdx.x * kBlock + threadIdx.x, row = units.row(at);
  const uint32_t unit = at - row * units.per_row;
  const bool live = row < c.rows;
  const int64_t col = (int64_t)unit * N;
  float v[N];
  uint32_t m = 0;
  if (live) {
    load_row<T>(X + row * ldx, col, c.cols, 0.0f, v);
#pragma unroll
    for (int e = 0; e < N; ++e) m = max(m, abs_bits(v[e]));
  }
  m = lanes_max_u32<LANES>(m);                            // a group's lanes are one aligned run of lanes
  if (!live) return;
  const float s = scale_of_bits(m);
  const float inv = recip_rn(s);
  const bool fine = m < kInfBits;
  int q[N];
#pragma unroll
  for (int e = 0; e < N; ++e) q[e] = fine ? quantize1(v[e], inv) : 0;
  store_codes(c.Q + row * c.ldq, col, c.cols, q);
  if (unit % LANES == 0) c.scale[row * c.lds + unit / LANES] = s;
}

// The derivative of GELU in its tanh form: with v = 2 sqrt(2/pi) (x + 0.044715
// x^3) and p = 1/(1 + exp(-v)),
//   gelu(x) = x p,   gelu'(x) = p + x v' p (1-p).
// With z = exp(-|v|) and d = 1/(1+z), the two of p and 1-p are d and z d.
// Beyond |x| = 10 the derivative is within 3e-36 of 0 or 1, so x is kept to
// that range and z above 2^-126.
__device__ __forceinline__ float gelu_grad(float x) {
  x = __builtin_amdgcn_fmed3f(x, -10.0f, 10.0f);
  const float x2 = x * x, cx = 1.59576912f * x;
  const float v = cx * __builtin_fmaf(0.044715f, x2, 1.0f);
  const float z = exp_small(-fabsf(v));
  const float d = recip_1_2(1.0f + z), zd = z * d;
  const float xv = cx * __builtin_fmaf(0.134145f, x2, 1.0f);
  return __builtin_fmaf(xv, zd * d, v < 0.0f ? zd : d);
}

template <class T, int ACT>
__global__ void __launch_bounds__(kBlock) checkpoint_read_kernel(Checkpoint c, const T* __restrict__ dY, int64_t lddy,
                                                                 T* __restrict__ Y, int64_t ldy, Units units) {
  constexpr int N = kVec<T>;
  const uint32_t at = blockIdx.x * kBlock + threadIdx.x, row = units.row(at);
  if (row >= c.rows) return;
  const int64_t col = (int64_t)(at - row * units.per_row) * N;
  int q[N];
  load_codes(c.Q + row * c.ldq, col, c.cols, q);
  const float s = c.scale[row * c.lds + (col >> c.gshift)];
  float y[N];
  if constexpr (ACT != ACT_NONE) load_row<T>(dY + row * lddy, col, c.cols, 0.0f, y);
  const float nan = s - s;                                // 0, or NaN with the scale
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float x = mul_rn((float)q[e], s);
    if constexpr (ACT == ACT_NONE) y[e] = x;
    if constexpr (ACT == ACT_RELU) y[e] = x > 0.0f ? y[e] : nan;
    if constexpr (ACT == ACT_GELU) y[e] = y[e] * (gelu_grad(x) + nan);
  }
  store_row<T>(Y + row * ldy, col, c.cols, y);
}

// ---------------------------------------------------------------------------
// quantize_cols of a checkpoint's values: a pass for the column scales (the
// largest partial scale is the scale of the column's maximum, as rounding is
// monotone, so atomicMax on the bits of the scales is exact in any order; a
// NaN is the largest), then a pass that quantizes and transposes.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) checkpoint_cols_init_kernel(float* scale, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) scale[i] = scale_floor();
}

constexpr int kColRows = 64;     // rows of a workgroup of the scale pass

__global__ void __launch_bounds__(256) checkpoint_cols_scale_kernel(Checkpoint c, unsigned int* __restrict__ scale) {
  __shared__ uint32_t red[4][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 256 + lane * 4;
  for (int64_t r0 = (int64_t)blockIdx.y * kColRows; r0 < c.rows; r0 += (int64_t)gridDim.y * kColRows) {
    uint32_t m[4] = {0, 0, 0, 0};
    if (col < c.cols) {
      const int64_t end = r0 + kColRows < c.rows ? r0 + kColRows : c.rows;
      for (int64_t r = r0 + wave; r < end; r += 4) {
        int q[4];
        load_codes(c.Q + r * c.ldq, col, c.cols, q);
        const float s = c.scale[r * c.lds + (col >> c.gshift)];
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = max(m[e], abs_bits(mul_rn((float)q[e], s)));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][lane * 4 + e] = m[e];
    __syncthreads();
    const int t = threadIdx.x;
    const uint32_t a = max(max(red[0][t], red[1][t]), max(red[2][t], red[3][t]));
    if ((int64_t)blockIdx.x * 256 + t < c.cols)
      atomicMax(scale + (int64_t)blockIdx.x * 256 + t, __float_as_uint(scale_of_bits(a)));
    __syncthreads();
  }
}

// 64 rows x 64 columns: quantized, transposed through LDS, stored as 64 rows
// of 64 bytes.
__global__ void __launch_bounds__(256) checkpoint_cols_quant_kernel(Checkpoint c, int8_t* __restrict__ Qt,
                                                                    int64_t ldqt, const float* __restrict__ scale) {
  __shared__ float s_inv[64];
  __shared__ unsigned int tile[64][17];
  const int tid = threadIdx.x;
  const int64_t j0 = (int64_t)blockIdx.x * 64;
  if (tid < 64) {
    const float s = j0 + tid < c.cols ? scale[j0 + tid] : 1.0f;
    s_inv[tid] = s == s ? recip_rn(s) : 0.0f;             // a NaN column: codes 0
  }
  __syncthreads();
  const int cg = tid & 15, rr = tid >> 4;
  const int64_t col = j0 + cg * 4;
  float inv[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) inv[e] = s_inv[cg * 4 + e];
  for (int64_t k0 = (int64_t)blockIdx.y * 64; k0 < c.rows; k0 += (int64_t)gridDim.y * 64) {
    unsigned int w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = k0 + rr * 4 + i;
      if (k < c.rows && col < c.cols) {
        int q[4];
        load_codes(c.Q + k * c.ldq, col, c.cols, q);
        const float s = c.scale[k * c.lds + (col >> c.gshift)];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = inv[e] > 0.0f ? quantize1(mul_rn((float)q[e], s), inv[e]) : 0;
          w[e] |= (unsigned int)(v & 0xFF) << (8 * i);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) tile[cg * 4 + e][rr] = w[e];
    __syncthreads();
    const int jl = tid >> 2, ch = tid & 3;
    const int64_t j = j0 + jl, k = k0 + ch * 16;
    if (j < c.cols && k < c.rows) {
      int8_t* dst = Qt + j * ldqt + k;
      unsigned int t[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = tile[jl][ch * 4 + e];
      if (k + 16 <= c.rows) {
        __builtin_memcpy(dst, t, 16);
      } else {
        for (int e = 0; e < 16 && k + e < c.rows; ++e) dst[e] = (int8_t)((t[e >> 2] >> (8 * (e & 3))) & 0xFF);
      }
    }
    __syncthreads();
  }
}

// Calls launch(first row, rows, grid) for slabs of rows of fewer than 2^31 units.
template <class F>
void for_slabs(int64_t rows, const Units& u, F launch) {
  const int64_t most = ((int64_t(1) << 31) - kBlock) / u.per_row;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = rows - r < most ? rows - r : most;
    launch(r, n, dim3((unsigned int)((n * u.per_row + kBlock - 1) / kBlock)));
  }
}

Checkpoint slab_of(Checkpoint c, int64_t first, int64_t rows) {
  c.Q += first * c.ldq;
  c.scale += first * c.lds;
  c.rows = rows;
  return c;
}

template <class T, int GROUP>
hipError_t store(const T* x, int64_t ldx, const Checkpoint& c, hipStream_t stream) {
  const Units u = units_of(c.cols, GROUP, kVec<T>);
  for_slabs(c.rows, u, [&](int64_t first, int64_t rows, dim3 grid) {
    hipLaunchKernelGGL((checkpoint_store_kernel<T, GROUP>), grid, dim3(kBlock), 0, stream, x + first * ldx, ldx,
                       slab_of(c, first, rows), u);
  });
  return hipGetLastError();
}

template <class T>
hipError_t store(const void* X, int64_t ldx, const Checkpoint& c, hipStream_t stream) {
  const T* x = static_cast<const T*>(X);
  switch (1 << c.gshift) {
    case 32: return store<T, 32>(x, ldx, c, stream);
    case 64: return store<T, 64>(x, ldx, c, stream);
    case 128: return store<T, 128>(x, ldx, c, stream);
    default: return store<T, 256>(x, ldx, c, stream);
  }
}

template <class T, int ACT>
hipError_t read(const Checkpoint& c, const T* dy, int64_t lddy, T* y, int64_t ldy, hipStream_t stream) {
  const Units u = units_of(c.cols, kVec<T>, kVec<T>);
  for_slabs(c.rows, u, [&](int64_t first, int64_t rows, dim3 grid) {
    hipLaunchKernelGGL((checkpoint_read_kernel<T, ACT>), grid, dim3(kBlock), 0, stream, slab_of(c, first, rows),
                       dy ? dy + first * lddy : dy, lddy, y + first * ldy, ldy, u);
  });
  return hipGetLastError();
}

template <class T>
hipError_t read(const Checkpoint& c, int act, const void* dY, int64_t lddy, void* Y, int64_t ldy, hipStream_t stream) {
  const T* dy = static_cast<const T*>(dY);
  T* y = static_cast<T*>(Y);
  switch (act) {
    case ACT_NONE: return read<T, ACT_NONE>(c, dy, lddy, y, ldy, stream);
    case ACT_RELU: return read<T, ACT_RELU>(c, dy, lddy, y, ldy, stream);
    default: return read<T, ACT_GELU>(c, dy, lddy, y, ldy, stream);
  }
}

}  // namespace

hipError_t launch_checkpoint_store(const void* X, int64_t ldx, int dtype, const Checkpoint& c, hipStream_t stream) {
  switch (dtype) {
    case DT_F32: return store<float>(X, ldx, c, stream);
    case DT_BF16: return store<bf16_t>(X, ldx, c, stream);
    default: return store<f16_t>(X, ldx, c, stream);
  }
}

hipError_t launch_checkpoint_read(const Checkpoint& c, int act, const void* dY, int64_t lddy, void* Y, int64_t ldy,
                                  int dtype, hipStream_t stream) {
  switch (dtype) {
    case DT_F32: return read<float>(c, act, dY, lddy, Y, ldy, stream);
    case DT_BF16: return read<bf16_t>(c, act, dY, lddy, Y, ldy, stream);
    default: return read<f16_t>(c, act, dY, lddy, Y, ldy, stream);
  }
}

hipError_t launch_checkpoint_cols(const Checkpoint& c, int8_t* Qt, int64_t ldqt, float* scale, hipStream_t stream) {
  hipLaunchKernelGGL(checkpoint_cols_init_kernel, dim3((unsigned int)((c.cols + 255) / 256)), dim3(256), 0, stream,
                     scale, c.cols);
  if (c.rows > 0) {
    const int64_t by = (c.rows + 63) / 64;
    const unsigned int gy = (unsigned int)(by < 4096 ? by : 4096);
    hipLaunchKernelGGL(checkpoint_cols_scale_kernel, dim3((unsigned int)((c.cols + 255) / 256), gy), dim3(256), 0,
                       stream, c, reinterpret_cast<unsigned int*>(scale));
    hipLaunchKernelGGL(checkpoint_cols_quant_kernel, dim3((unsigned int)((c.cols + 63) / 64), gy), dim3(256), 0,
                       stream, c, Qt, ldqt, scale);
  }
  return hipGetLastError();
}

}  // namespace i8g
