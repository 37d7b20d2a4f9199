// checkpoint.hip -- activation checkpoints in 8 bits and their use in the
// backward pass.  A checkpoint is the quantize_rows rule applied to each
// group of 32 to 256 columns of a row: s = max(RN(a/127), RN(1e-8)),
// q = floor(RN(RN(x*RN(1/s)) + 0.5)), and stands for RN(q*s).  A group that
// holds an infinity or a NaN gets a NaN scale, so it restores as NaN.
//
// Storing reads a value and writes a byte; restoring, the activation's
// gradient and the column quantization of a checkpoint read that byte where
// they would have read a value.  They are bound by memory: 8192 x 3072 f32 in
// groups of 128 is stored in 20.4 us and restored in 19.8 (126 MB each, 6.2
// and 6.4 TB/s; a copy within the 256 MB cache moves 6.9), the gradient of GELU
// in bf16 takes 24.2 us (126 MB, 5.2 TB/s; its 42 instructions a value are next).
// The column quantization's two passes are bound by latency, a thread having
// four 8-byte loads in flight: 5.2 and 8.0 us for 8192 x 768, of which the
// launch and the first load are 2 each, and 11.1 and 17.6 us for 8192 x 3072
// (2.3 and 2.9 TB/s).
#include <type_traits>

#include "i8g_launch.h"
#include "i8g_row.h"

namespace i8g {
namespace {

constexpr int kBlock = 256;

// The division of a number below 2^31 by d as one multiplication: with
// 2^(l-1) < d <= 2^l and m = floor(2^(31+l) / d) + 1, n m / 2^(31+l) exceeds
// n / d by less than 1/d for n < 2^31, and its floor is exact.
struct Divisor {
  uint32_t d, mul, shift;
  __host__ explicit Divisor(uint32_t d) : d(d) {
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    shift = 31 + l;
    mul = (uint32_t)((uint64_t(1) << shift) / d + 1);
  }
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return (uint32_t)((uint64_t)n * mul >> shift); }
};

// The units of N columns of a matrix's rows are numbered row by row, and a
// lane takes one, so short and odd rows leave no lanes idle.  A launch covers
// fewer than 2^31 units; more rows take more launches.  (A wave on 64 units
// of 4 rows, which shares a row's addresses and lets every lane find one
// row's scale, stores 8192 x 3072 f32 2% faster, bf16 8% slower, and 2^20
// rows of 32 columns in twice the time.)
template <int N>
struct Place {
  uint32_t row, unit;
  int64_t col;
  __device__ __forceinline__ explicit Place(const Divisor& units) {
    const uint32_t n = blockIdx.x * kBlock + threadIdx.x;
    row = units.of(n);
    unit = n - row * units.d;
    col = (int64_t)unit * N;
  }
};

// Values of a lane of the store: its group's two divisions serve 8 values in
// f32 too (two 16-byte loads; 4 take 24.4 us for 8192 x 3072, 8 take 20.8).
constexpr int kStoreUnit = 8;

template <class T, int GROUP>
__global__ void __launch_bounds__(kBlock) checkpoint_store_kernel(const T* __restrict__ X, int64_t ldx, Checkpoint c,
                                                                  Divisor units) {
  constexpr int N = kStoreUnit, LANES = GROUP / N;        // a group's lanes are one aligned run of lanes
  const Place<N> at(units);
  const bool live = at.row < c.rows;
  float v[N];
  uint32_t m = 0;
  if (live) {
    load_row<T>(X + at.row * ldx, at.col, c.cols, 0.0f, v);
#pragma unroll
    for (int e = 0; e < N; ++e) m = max(m, abs_bits(v[e]));
  }
  m = lanes_max_u32<LANES>(m);
  if (!live) return;
  const float s = scale_of_bits(m);
  const float inv = recip_rn(s);
  const bool fine = m < kInfBits;
  int q[N];
#pragma unroll
  for (int e = 0; e < N; ++e) q[e] = fine ? quantize1(v[e], inv) : 0;
  store_codes(c.Q + at.row * c.ldq, at.col, c.cols, q);
  if (at.unit % LANES == 0) c.scale[at.row * c.lds + at.unit / LANES] = s;
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

// APART: Y shares nothing with dY; else it is dY itself, and no load of one
// value may be moved behind another's store.
template <class P, bool APART>
using Values = std::conditional_t<APART, P* __restrict__, P*>;

template <class T, int ACT, bool APART>
__global__ void __launch_bounds__(kBlock) checkpoint_read_kernel(Checkpoint c, Values<const T, APART> dY, int64_t lddy,
                                                                 Values<T, APART> Y, int64_t ldy, Divisor units) {
  constexpr int N = kVec<T>;
  const Place<N> at(units);
  if (at.row >= c.rows) return;
  CodeWords<N> q;
  q.load(c.Q + at.row * c.ldq, at.col, c.cols);
  const float s = c.scale[at.row * c.lds + (at.col >> c.gshift)];
  float y[N];
  if constexpr (ACT != ACT_NONE) load_row<T>(dY + at.row * lddy, at.col, c.cols, 0.0f, y);
  const float nan = s - s;                                // 0, or NaN with the scale
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float x = mul_rn(q[e], s);
    if constexpr (ACT == ACT_NONE) y[e] = x;
    if constexpr (ACT == ACT_RELU) y[e] = x > 0.0f ? y[e] : nan;
    if constexpr (ACT == ACT_GELU) y[e] = y[e] * (gelu_grad(x) + nan);
  }
  store_row<T>(Y + at.row * ldy, at.col, c.cols, y);
}

// ---------------------------------------------------------------------------
// quantize_cols of a checkpoint's values: a pass that leaves the column maxima
// of up to kColParts ranges of rows in the workspace, then a pass that takes
// the largest of them, quantizes and transposes.  Both work on tiles of 64
// columns x 128 rows, a thread on 8 columns (one 8-byte load a row, inside
// one group) of 4 rows.
// ---------------------------------------------------------------------------
constexpr int kTileCols = 64, kTileRows = 128;
constexpr int kColParts = 64;

// The values of columns col .. col+7 of 4 rows from `row`; 0 outside the
// matrix.  `inside`: the whole tile lies in the matrix.
__device__ __forceinline__ void tile_rows(const Checkpoint& c, int64_t row, int64_t col, bool inside,
                                          float (&v)[4][8]) {
  CodeWords<8> q[4];
  float s[4];
  const int8_t* Q = c.Q + row * c.ldq + col;
  const float* S = c.scale + row * c.lds + (col >> c.gshift);
  if (inside) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __builtin_memcpy(q[i].w, Q + i * c.ldq, 8);
      s[i] = S[i * c.lds];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool some = row + i < c.rows && col < c.cols;
      q[i].load(Q + i * c.ldq, (int64_t)0, some ? c.cols - col : (int64_t)0);
      s[i] = some ? S[i * c.lds] : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = mul_rn(q[i][e], s[i]);
}

// The largest of x over the lanes of equal number mod 8.
__device__ __forceinline__ uint32_t max_mod8(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, x, 0x128, 0xF, 0xF, true));   // rotated by 8 lanes of 16
  Pair32 p = lane_pair<16>(x);
  p = lane_pair<32>(max(p.a, p.b));
  return max(p.a, p.b);
}

// Column maxima, as the bits of |x| (a NaN is above all), of the row tiles
// blockIdx.y, blockIdx.y + gridDim.y, ...
__global__ void __launch_bounds__(256) checkpoint_cols_max_kernel(Checkpoint c, uint32_t* __restrict__ parts) {
  __shared__ uint32_t red[4][kTileCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * kTileCols + (threadIdx.x & 7) * 8;
  const bool wide = ((int64_t)blockIdx.x + 1) * kTileCols <= c.cols;
  uint32_t m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t r0 = (int64_t)blockIdx.y * kTileRows; r0 < c.rows; r0 += (int64_t)gridDim.y * kTileRows) {
    float v[4][8];
    tile_rows(c, r0 + (threadIdx.x >> 3) * 4, col, wide && r0 + kTileRows <= c.rows, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      m[e] = max(max(m[e], max(abs_bits(v[0][e]), abs_bits(v[1][e]))), max(abs_bits(v[2][e]), abs_bits(v[3][e])));
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m[e] = max_mod8(m[e]);
    if (lane < 8) red[wave][lane * 8 + e] = m[e];
  }
  __syncthreads();
  if (threadIdx.x < kTileCols)                            // rows of parts are whole tiles
    parts[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kTileCols + threadIdx.x] =
        max(max(red[0][threadIdx.x], red[1][threadIdx.x]), max(red[2][threadIdx.x], red[3][threadIdx.x]));
}

// Quantized, transposed through LDS (4 rows of a column to a word; a row of
// 33 words puts the 64 lanes of a wave on 64 banks) and stored as 64 rows of
// 128 bytes.  The workgroups of the first row tile write the scales.
__global__ void __launch_bounds__(256) checkpoint_cols_quant_kernel(Checkpoint c, int8_t* __restrict__ Qt,
                                                                    int64_t ldqt, float* __restrict__ scale,
                                                                    const uint32_t* __restrict__ parts, int n_parts) {
  __shared__ uint32_t red[4][kTileCols];
  __shared__ float s_inv[kTileCols];
  __shared__ unsigned int tile[kTileCols][kTileRows / 4 + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t j0 = (int64_t)blockIdx.x * kTileCols;
  const int cg = tid & 7, rr = tid >> 3;
  const int64_t col = j0 + cg * 8;
  int64_t r0 = (int64_t)blockIdx.y * kTileRows;
  float v[4][8];
  const bool wide = j0 + kTileCols <= c.cols;
  tile_rows(c, r0 + rr * 4, col, wide && r0 + kTileRows <= c.rows, v);   // on their way while the scales are found
  // the maxima of the row ranges, 4 columns a lane and 4 ranges a wave at a time
  uint32_t m[4] = {0, 0, 0, 0};
  for (int p = wave * 4 + (lane >> 4); p < n_parts; p += 16) {
    uint32_t x[4];
    __builtin_memcpy(x, parts + ((int64_t)p * gridDim.x + blockIdx.x) * kTileCols + (lane & 15) * 4, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = max(m[e], x[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    Pair32 p = lane_pair<16>(m[e]);
    p = lane_pair<32>(max(p.a, p.b));
    if (lane < 16) red[wave][lane * 4 + e] = max(p.a, p.b);
  }
  __syncthreads();
  if (tid < kTileCols) {
    const uint32_t a = max(max(red[0][tid], red[1][tid]), max(red[2][tid], red[3][tid]));
    const float s = scale_of_bits(a);
    s_inv[tid] = a < kInfBits ? recip_rn(s) : 0.0f;       // a NaN column: codes 0
    if (blockIdx.y == 0 && j0 + tid < c.cols) scale[j0 + tid] = s;
  }
  __syncthreads();
  float inv[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) inv[e] = s_inv[cg * 8 + e];
  while (r0 < c.rows) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned int w = pack_bytes(quantize1(v[0][e], inv[e]), quantize1(v[1][e], inv[e]),
                                        quantize1(v[2][e], inv[e]), quantize1(v[3][e], inv[e]));
      tile[cg * 8 + e][rr] = inv[e] > 0.0f ? w : 0u;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {                         // 8 threads store a column's 128 bytes
      const int jl = i * 32 + (tid >> 3), part = tid & 7;
      const int64_t j = j0 + jl, k = r0 + part * 16;
      if (j < c.cols && k < c.rows) {
        int8_t* dst = Qt + j * ldqt + k;
        unsigned int w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = tile[jl][part * 4 + e];
        if (k + 16 <= c.rows) {
          __builtin_memcpy(dst, w, 16);
        } else {
          for (int e = 0; e < 16 && k + e < c.rows; ++e) dst[e] = (int8_t)((w[e >> 2] >> (8 * (e & 3))) & 0xFF);
        }
      }
    }
    r0 += (int64_t)gridDim.y * kTileRows;
    if (r0 < c.rows) tile_rows(c, r0 + rr * 4, col, wide && r0 + kTileRows <= c.rows, v);
    __syncthreads();
  }
}

// The scales of columns without rows: the floor.
__global__ void __launch_bounds__(256) checkpoint_cols_floor_kernel(float* scale, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) scale[i] = scale_floor();
}

int64_t row_tiles(int64_t rows) { return (rows + kTileRows - 1) / kTileRows; }

// Calls launch(first row, rows, grid, divisor) for slabs of rows of fewer than
// 2^31 units; a row takes `units` of them.
template <class F>
void for_slabs(int64_t rows, int64_t units, F launch) {
  const Divisor d((uint32_t)units);
  const int64_t most = ((int64_t(1) << 31) - kBlock) / units;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = rows - r < most ? rows - r : most;
    launch(r, n, dim3((unsigned int)((n * units + kBlock - 1) / kBlock)), d);
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
  const int64_t units = (c.cols + GROUP - 1) / GROUP * (GROUP / kStoreUnit);  // whole groups
  for_slabs(c.rows, units, [&](int64_t first, int64_t rows, dim3 grid, const Divisor& d) {
    hipLaunchKernelGGL((checkpoint_store_kernel<T, GROUP>), grid, dim3(kBlock), 0, stream, x + first * ldx, ldx,
                       slab_of(c, first, rows), d);
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

template <class T, int ACT, bool APART>
hipError_t read(const Checkpoint& c, const T* dy, int64_t lddy, T* y, int64_t ldy, hipStream_t stream) {
  for_slabs(c.rows, (c.cols + kVec<T> - 1) / kVec<T>, [&](int64_t first, int64_t rows, dim3 grid, const Divisor& d) {
    hipLaunchKernelGGL((checkpoint_read_kernel<T, ACT, APART>), grid, dim3(kBlock), 0, stream, slab_of(c, first, rows),
                       dy ? dy + first * lddy : dy, lddy, y + first * ldy, ldy, d);
  });
  return hipGetLastError();
}

// The instance that is right in place leaves the compiler less freedom: on
// matrices apart, GELU's gradient of 8192 x 3072 bf16 takes 28.3 us with it and
// 25.3 with the other.  (ReLU's and f32 take the same.)
template <class T, int ACT>
hipError_t read(const Checkpoint& c, const T* dy, int64_t lddy, T* y, int64_t ldy, hipStream_t stream) {
  return dy == y ? read<T, ACT, false>(c, dy, lddy, y, ldy, stream) : read<T, ACT, true>(c, dy, lddy, y, ldy, stream);
}

template <class T>
hipError_t read(const Checkpoint& c, int act, const void* dY, int64_t lddy, void* Y, int64_t ldy, hipStream_t stream) {
  const T* dy = static_cast<const T*>(dY);
  T* y = static_cast<T*>(Y);
  switch (act) {
    case ACT_NONE: return read<T, ACT_NONE, true>(c, dy, lddy, y, ldy, stream);
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

static int cols_parts(int64_t rows) {
  const int64_t n = row_tiles(rows);
  return (int)(n < kColParts ? n : kColParts);
}

size_t checkpoint_cols_words(int64_t rows, int64_t cols) {
  return (size_t)cols_parts(rows) * ((cols + kTileCols - 1) / kTileCols * kTileCols);
}

hipError_t launch_checkpoint_cols(const Checkpoint& c, int8_t* Qt, int64_t ldqt, float* scale, void* parts,
                                  hipStream_t stream) {
  if (c.rows == 0) {
    hipLaunchKernelGGL(checkpoint_cols_floor_kernel, dim3((unsigned int)((c.cols + 255) / 256)), dim3(256), 0, stream,
                       scale, c.cols);
    return hipGetLastError();
  }
  uint32_t* p = static_cast<uint32_t*>(parts);
  const int n = cols_parts(c.rows);
  const int64_t tiles = row_tiles(c.rows);
  // a launch holds fewer than 2^32 threads, 4 a column; slabs of columns are whole groups
  const int64_t slab = int64_t(1) << 29;
  for (int64_t j = 0; j < c.cols; j += slab) {
    Checkpoint part = c;
    part.Q += j;
    part.scale += j >> c.gshift;
    part.cols = c.cols - j < slab ? c.cols - j : slab;
    const unsigned int bx = (unsigned int)((part.cols + kTileCols - 1) / kTileCols);
    hipLaunchKernelGGL(checkpoint_cols_max_kernel, dim3(bx, n), dim3(256), 0, stream, part, p);
    hipLaunchKernelGGL(checkpoint_cols_quant_kernel, dim3(bx, (unsigned int)(tiles < 4096 ? tiles : 4096)), dim3(256),
                       0, stream, part, Qt + j * ldqt, ldqt, scale + j, p, n);
  }
  return hipGetLastError();
}

}  // namespace i8g
