// logprob.hip -- log probabilities of given tokens from a matrix of logits,
// with the entropy and the best alternatives of every row, and the gradient.
//
// For a row x of V logits, with M = max x, S = sum exp(x - M) and
// T = sum exp(x - M) (x - M):
//   lse = M + log S     log p_j = x_j - M - log S     H = log S - T / S
//   dx_j = g ([j = t] - p_j) - gH p_j (log p_j + H)
// One pass over the logits: a thread keeps the running maximum of its values
// and its two sums against that maximum (binary32, at most 128 values), which
// are rescaled when the maximum grows; threads and parts are joined in
// binary64.  Both directions are bound by reading the logits (and writing the
// gradient); the exponential's ~20 operations a value are next.
#include "i8g_launch.h"
#include "i8g_row.h"

namespace i8g {
namespace {

constexpr int kThreads = 512;                 // of a workgroup of the forward pass
constexpr int kValues = 128;                  // values of a thread at most
constexpr int kSegMax = kThreads * kValues;   // columns of a part at most
constexpr int kMaxParts = 64;                 // parts of a row at most (a wave joins them)
constexpr int kTopMax = 32;
constexpr float kLowest = -3.40282347e38f;    // the running maximum's start: finite, so x - m is never NaN for finite x or -inf

struct PartSum {
  double s, t;
  float m;
};

// An integer that orders like x (-0 and +0 alike, NaN with -inf); 0 is below
// every value.
__device__ __forceinline__ uint32_t rank_key(float x) {
  if (x != x) return 0x00800000u;
  const uint32_t b = __float_as_uint(x);
  const int o = (int)b < 0 ? -(int)(b & 0x7FFFFFFFu) : (int)b;
  return (uint32_t)o ^ 0x80000000u;
}
__device__ __forceinline__ float rank_value(uint32_t key) {
  const int o = (int)(key ^ 0x80000000u);
  return __uint_as_float(o < 0 ? (uint32_t)(-o) | 0x80000000u : (uint32_t)o);
}
// The largest of a wave's (never NaN) values.
__device__ __forceinline__ float wave_max(float x) { return rank_value(lanes_max_u32<64>(rank_key(x))); }
// Larger for the larger value, then for the lower index.
__device__ __forceinline__ uint64_t candidate(uint32_t key, uint32_t index) {
  return (uint64_t)key << 32 | (0xFFFFFFFFu - index);
}

// (s, t) against the maximum `from`, rescaled to the larger maximum `to`.
__device__ __forceinline__ void rescale(float& s, float& t, float from, float to) {
  const float d = __builtin_elementwise_maximum(from - to, -104.0f);
  const float f = exp_f32(d);
  t = f * (t + s * d);
  s = f * s;
}

// The outputs of one row from its joined sums (one thread).
struct RowOut {
  double m, log_s;
  bool empty;                                 // no value above -inf
  __device__ __forceinline__ RowOut(const PartSum& p) : m(p.m), log_s(log(p.s)), empty(p.s == 0.0) {}
  __device__ __forceinline__ float log_prob(float x) const {
    return empty ? -__builtin_inff() : (float)((double)x - m - log_s);
  }
};

template <class T>
__device__ __forceinline__ void write_row(const LpArgs& a, int64_t r, const PartSum& p, const RowOut& o) {
  if (a.lse) a.lse[r] = o.empty ? -__builtin_inff() : (float)(o.m + o.log_s);
  if (a.entropy) {
    const double h = o.log_s - p.t / p.s;
    a.entropy[r] = o.empty ? 0.0f : h < 0.0 ? 0.0f : (float)h;
  }
  if (a.logprob) {
    const int64_t t = a.targets[r];
    const bool given = t >= 0 && t < a.cols;
    a.logprob[r] = given ? o.log_prob(to_f32(static_cast<const T*>(a.X)[r * a.ldx + t])) : 0.0f;
  }
}

// The k best of n candidates in LDS, best first: a candidate's place is the
// number of better ones.  Four lanes count for each, 8 at a time so that the
// reads overlap, until they know that it is not among the best.  `list` has
// room for kPad more, which the caller has set to 0 (pad_list).
constexpr int kPad = 31;
__device__ __forceinline__ void pad_list(unsigned long long* list, int n) {
  if (threadIdx.x < kPad) list[n + threadIdx.x] = 0;
}
__device__ __forceinline__ void place_best(const unsigned long long* list, int n, int k, unsigned long long* best,
                                           int thread, int threads) {
  const int part = thread & 3;
  for (int i = thread >> 2; i < n; i += threads >> 2) {
    const unsigned long long mine = list[i];
    int above = 0;
    for (int j = part * 8; j < n && above < k; j += 32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) above += list[j + e] > mine ? 1 : 0;
    }
    above += lane_partner<1>(above);
    above += lane_partner<2>(above);
    if (part == 0 && above < k && mine != 0) best[above] = mine;
  }
}

// LDS of the search for the best alternatives.
struct TopLds {
  uint32_t key[kThreads];                     // the largest key of each thread
  unsigned long long list[(kTopMax - 1) * kValues + 1024 + kPad];
  unsigned long long best[kTopMax];
  int lane_of[kTopMax - 1 + 32];
  int wave_count[kThreads / 64];
  uint32_t bar;
  int n_above, n_equal, n_cand, n_cand_equal;
};

// The min(k, values) best of a part's values into l.best (unused places 0).
// The k-th largest of the threads' maxima is a bar that at least k values
// reach, and values above it are only in the fewer than k threads whose
// maximum is above it: those threads' values are read again (from cache),
// with those of the threads whose maximum is the bar itself.  If that many
// values equal the bar that they would not fit (masked rows), the ones of
// lowest index are found by a scan from the part's start.
template <class T>
__device__ __forceinline__ void find_best(TopLds& l, const T* row, int lo, int hi, float mx, int k) {
  constexpr int N = kVec<T>, NV = kValues / N;
  constexpr int kAbove = (kTopMax - 1) * kValues;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t mine = rank_key(mx);
  l.key[tid] = mine;
  if (tid < kTopMax) l.best[tid] = 0;
  if (tid == 0) l.n_above = l.n_equal = l.n_cand = l.n_cand_equal = 0;
  __syncthreads();
  if (wave == 0) {                            // the largest bar that k threads reach, bit by bit
    uint32_t key[kThreads / 64];
#pragma unroll
    for (int j = 0; j < kThreads / 64; ++j) key[j] = l.key[lane + 64 * j];
    uint32_t bar = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t b = bar | 1u << bit;
      int n = 0;
#pragma unroll
      for (int j = 0; j < kThreads / 64; ++j) n += __popcll(__ballot(key[j] >= b));
      if (n >= k) {
        bar = b;
        if (n == k) break;
      }
    }
    if (lane == 0) l.bar = bar;
  }
  __syncthreads();
  const uint32_t bar = l.bar;
  if (mine > bar) l.lane_of[atomicAdd(&l.n_above, 1)] = tid;      // fewer than k
  __syncthreads();
  const int n_above = l.n_above;
  if (mine == bar) {
    const int i = atomicAdd(&l.n_equal, 1);
    if (i < 32) l.lane_of[n_above + i] = tid;
  }
  __syncthreads();
  const bool few = l.n_equal <= 32;
  const int n_lanes = n_above + (few ? l.n_equal : 0);
  for (int i = tid / NV; i < n_lanes; i += kThreads / NV) {       // NV lanes read a thread's vectors
    const int c = lo + (l.lane_of[i] + kThreads * (tid % NV)) * N;
    if (c >= hi) continue;
    float v[N];
    load_row<T>(row, c, hi, 0.0f, v);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (c + e >= hi) continue;
      const uint32_t key = rank_key(v[e]);
      if (key > bar) {
        l.list[atomicAdd(&l.n_cand, 1)] = candidate(key, c + e);
      } else if (key == bar) {
        const int at = atomicAdd(&l.n_cand_equal, 1);
        if (at < 1024) l.list[kAbove + at] = candidate(key, c + e);
      }
    }
  }
  __syncthreads();
  int n = l.n_cand, n_eq = l.n_cand_equal;
  if (n >= k) n_eq = 0;
  if (n < k && (!few || n_eq > 1024)) {
    // the values that equal the bar, from the part's start
    const int need = k - n;
    n_eq = 0;
    for (int base = lo; base < hi && n_eq < need; base += kThreads * N) {
      const int c = base + tid * N;
      float v[N];
      unsigned int hit = 0;
      if (c < hi) {
        load_row<T>(row, c, hi, 0.0f, v);
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (c + e < hi && rank_key(v[e]) == bar) hit |= 1u << e;
      }
      int before = __popc(hit);               // inclusive sum over the lanes, then exclusive
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(before, off, 64);
        if (lane >= off) before += o;
      }
      if (lane == 63) l.wave_count[wave] = before;
      before -= __popc(hit);
      __syncthreads();
      int total = 0;
      for (int w = 0; w < kThreads / 64; ++w) {
        if (w < wave) before += l.wave_count[w];
        total += l.wave_count[w];
      }
      before += n_eq;
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (hit >> e & 1u) {
          if (before < need) l.list[kAbove + before] = candidate(bar, c + e);
          ++before;
        }
      n_eq += total;
      __syncthreads();
    }
    n_eq = n_eq < need ? n_eq : need;
  }
  // one list: the equal ones behind the ones above
  unsigned long long moved[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = tid + i * kThreads;
    moved[i] = at < n_eq ? l.list[kAbove + at] : 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = tid + i * kThreads;
    if (at < n_eq) l.list[n + at] = moved[i];
  }
  pad_list(l.list, n + n_eq);
  __syncthreads();
  place_best(l.list, n + n_eq, k, l.best, tid, kThreads);
  __syncthreads();
}

template <class T, bool TOP>
__global__ void __launch_bounds__(kThreads) lp_part_kernel(LpArgs a) {
  constexpr int N = kVec<T>, U = 16 / N;      // vectors of a batch: 16 values
  __shared__ double red_s[kThreads / 64], red_t[kThreads / 64];
  __shared__ float red_m[kThreads / 64];
  __shared__ __attribute__((aligned(16))) char top_bytes[TOP ? sizeof(TopLds) : 16];
  TopLds& top = *reinterpret_cast<TopLds*>(top_bytes);
  __shared__ double row_m, row_l;
  __shared__ int row_empty;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = blockIdx.x, lo = part * a.seg;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const int64_t task = r * a.parts + part;
    const int hi = lo + a.seg < a.cols ? lo + a.seg : (int)a.cols;
    const T* row = static_cast<const T*>(a.X) + r * a.ldx;
    float m = kLowest, mx = -__builtin_inff(), s = 0.0f, t = 0.0f;
    for (int base = lo; base < hi; base += kThreads * N * U) {
      float v[U][N];
#pragma unroll
      for (int u = 0; u < U; ++u) load_row<T>(row, base + (u * kThreads + tid) * N, hi, -__builtin_inff(), v[u]);
      float b = -__builtin_inff();
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) b = fmaxf(b, v[u][e]);
      mx = fmaxf(mx, b);
      if (b > m) {
        rescale(s, t, m, b);
        m = b;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float d = __builtin_elementwise_maximum(v[u][e] - m, -104.0f);   // (a NaN stays)
          const float p = exp_f32(d);
          s += p;
          t = __builtin_fmaf(p, d, t);
        }
    }
    // join the threads
    float mm = wave_max(m);
    if (lane == 0) red_m[wave] = mm;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) mm = fmaxf(mm, red_m[w]);
    rescale(s, t, m, mm);
    const double ws = wave_sum_f64((double)s), wt = wave_sum_f64((double)t);
    if (lane == 0) {
      red_s[wave] = ws;
      red_t[wave] = wt;
    }
    __syncthreads();
    PartSum p{0.0, 0.0, mm};
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
      p.s += red_s[w];
      p.t += red_t[w];
    }
    if (a.parts > 1) {
      if (tid == 0) a.sums[task] = LpPart{p.s, p.t, p.m, 0.0f};
      if constexpr (TOP) {
        find_best<T>(top, row, lo, hi, mx, a.topk);
        if (tid < a.topk) a.cands[task * a.topk + tid] = top.best[tid];
      }
    } else {
      if (tid == 0) {
        const RowOut o(p);
        write_row<T>(a, r, p, o);
        row_m = o.m;
        row_l = o.log_s;
        row_empty = o.empty;
      }
      if constexpr (TOP) {
        find_best<T>(top, row, lo, hi, mx, a.topk);
        if (tid < a.topk) {
          const unsigned long long c = top.best[tid];
          const float v = rank_value((uint32_t)(c >> 32));
          a.top_index[r * a.topk + tid] = (int32_t)(0xFFFFFFFFu - (uint32_t)c);
          a.top_logprob[r * a.topk + tid] = row_empty ? -__builtin_inff() : (float)((double)v - row_m - row_l);
        }
      }
    }
    __syncthreads();                          // LDS is used again
  }
}

// Joins the parts of a row: wave 0 their sums, the other waves their best.
constexpr int kJoinThreads = 1024;
template <class T>
__global__ void __launch_bounds__(kJoinThreads) lp_join_kernel(LpArgs a) {
  __shared__ unsigned long long list[kMaxParts * kTopMax + kPad];
  __shared__ unsigned long long best[kTopMax];
  __shared__ double row_m, row_l;
  __shared__ int row_empty;
  const int tid = threadIdx.x, n = a.parts * a.topk;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    for (int i = tid; i < n; i += kJoinThreads) list[i] = a.cands[r * n + i];
    pad_list(list, n);
    __syncthreads();
    if (tid < 64) {
      LpPart q{0.0, 0.0, kLowest, 0.0f};
      if (tid < a.parts) q = a.sums[r * a.parts + tid];
      const float mm = wave_max(q.m);
      double d = (double)q.m - (double)mm;
      d = d < -800.0 ? -800.0 : d;
      const double f = exp(d);
      PartSum p;
      p.t = wave_sum_f64(f * (q.t + q.s * d));
      p.s = wave_sum_f64(f * q.s);
      p.m = mm;
      if (tid == 0) {
        const RowOut o(p);
        write_row<T>(a, r, p, o);
        row_m = o.m;
        row_l = o.log_s;
        row_empty = o.empty;
      }
    } else {
      place_best(list, n, a.topk, best, tid - 64, kJoinThreads - 64);
    }
    __syncthreads();
    if (tid < a.topk) {
      const unsigned long long c = best[tid];
      const float v = rank_value((uint32_t)(c >> 32));
      a.top_index[r * a.topk + tid] = (int32_t)(0xFFFFFFFFu - (uint32_t)c);
      a.top_logprob[r * a.topk + tid] = row_empty ? -__builtin_inff() : (float)((double)v - row_m - row_l);
    }
    __syncthreads();                          // LDS is used again
  }
}

constexpr int kGradVecs = 4;                  // vectors of a thread of the backward pass

template <class T, bool STREAM>
__global__ void __launch_bounds__(256) lp_bwd_kernel(LpBwdArgs a) {
  constexpr int N = kVec<T>, U = kGradVecs;
  constexpr int CHUNK = 256 * N * U;
  const int64_t c0 = (int64_t)blockIdx.x * CHUNK + (int64_t)threadIdx.x * N;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const T* x = static_cast<const T*>(a.X) + r * a.ldx;
    T* dx = static_cast<T*>(a.dX) + r * a.lddx;
    const float lse = a.lse[r];
    int64_t t = a.g_logprob ? a.targets[r] : -1;
    if (t >= a.cols) t = -1;
    const float g = t >= 0 ? a.g_logprob[r] : 0.0f;
    const float gh = a.g_entropy ? a.g_entropy[r] : 0.0f;
    const float h = a.g_entropy ? a.entropy[r] : 0.0f;
    const bool empty = fabsf(lse) >= 16777216.0f;   // -inf, or so far out that lse is off by 1 and more
    float v[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) load_row<T>(x, c0 + u * 256 * N, a.cols, 0.0f, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 256 * N;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float lp = __builtin_elementwise_maximum(v[u][e] - lse, -104.0f);   // p is 0 there, and p * lp as well
        const float p = exp_f32(lp);
        float d = -p * (g + gh * (lp + h));
        if (c + e == t) d += g;
        v[u][e] = empty ? 0.0f : d;
      }
      if constexpr (STREAM)
        stream_row<T>(dx, c, a.cols, v[u]);
      else
        store_row<T>(dx, c, a.cols, v[u]);
    }
  }
}

// Rows are the grid's y; the workgroups walk on where there are more.
unsigned int row_grid(int64_t rows) { return (unsigned int)(rows < 65535 ? rows : 65535); }

template <class T>
hipError_t forward(const LpArgs& a, hipStream_t stream) {
  const dim3 grid(a.parts, row_grid(a.rows)), block(kThreads);
  if (a.topk > 0)
    hipLaunchKernelGGL((lp_part_kernel<T, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((lp_part_kernel<T, false>), grid, block, 0, stream, a);
  if (a.parts > 1) hipLaunchKernelGGL((lp_join_kernel<T>), dim3(1, row_grid(a.rows)), dim3(kJoinThreads), 0, stream, a);
  return hipGetLastError();
}

template <class T>
hipError_t backward(const LpBwdArgs& a, hipStream_t stream) {
  constexpr int CHUNK = 256 * kVec<T> * kGradVecs;
  const dim3 grid((unsigned int)((a.cols + CHUNK - 1) / CHUNK), row_grid(a.rows));
  // a gradient larger than half the last-level cache is stored around it
  if ((double)a.rows * (double)a.cols * sizeof(T) > kStreamOutBytes)
    hipLaunchKernelGGL((lp_bwd_kernel<T, true>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((lp_bwd_kernel<T, false>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

// Parts of a row: as many as its length needs, and with few rows as many as
// fill the chip, each of a batch of 16 values a thread (8192 columns) or more.
LpSplit lp_split(int64_t rows, int64_t cols) {
  int64_t parts = (cols + kSegMax - 1) / kSegMax;
  const int64_t fill = rows >= 512 ? 1 : (512 + rows - 1) / rows;
  int64_t most = (cols + 16 * kThreads - 1) / (16 * kThreads);
  most = most < kMaxParts ? most : kMaxParts;
  if (parts < fill) parts = fill < most ? fill : most > parts ? most : parts;
  const int64_t seg = ((cols + parts - 1) / parts + 63) / 64 * 64;
  return LpSplit{(int)((cols + seg - 1) / seg), (int)seg};
}

hipError_t launch_token_logprobs(const LpArgs& a, int dtype, hipStream_t stream) {
  switch (dtype) {
    case DT_F32: return forward<float>(a, stream);
    case DT_BF16: return forward<bf16_t>(a, stream);
    default: return forward<f16_t>(a, stream);
  }
}

hipError_t launch_token_logprobs_bwd(const LpBwdArgs& a, int dtype, hipStream_t stream) {
  switch (dtype) {
    case DT_F32: return backward<float>(a, stream);
    case DT_BF16: return backward<bf16_t>(a, stream);
    default: return backward<f16_t>(a, stream);
  }
}

}  // namespace i8g
