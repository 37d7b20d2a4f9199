// embedding.hip -- rows of a table looked up by token, and the table's
// gradient.
//
//   Y_i  = RN(alpha W[t_i]) + P[p_i]         W in f32, bf16, f16, or codes and scales: W = RN(q s)
//   dW_v = alpha sum_{t_i = v} dY_i          binary64 sums in the order of i
//
// The lookup is one pass: a wave takes up to 256 vectors of a row, four loads
// in flight.  The gradient sorts the tokens (a stable radix sort of 8192 at a
// time in LDS, while the other workgroups write the rows that no token names;
// the sorted runs are merged 8 at a time), then adds rows in the sorted order:
// a wave takes kPiece places of the order and a chunk of columns, writes the
// rows of tokens whose places it holds all of, and leaves the others' sums in
// the workspace, which a last launch joins.  No sum depends on which
// workgroup comes first.
#include "../../include/int8_gemm.h"
#include "i8g_launch.h"
#include "i8g_row.h"

#include <type_traits>

namespace i8g {
namespace {

template <class T>
__device__ __forceinline__ T uniform(T x) {
  static_assert(sizeof(T) == 4, "one register");
  return __builtin_bit_cast(T, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}
__device__ __forceinline__ int64_t uniform64(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)x >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// ---- lookup -----------------------------------------------------------------------
constexpr int kWaveVectors = 256;              // vectors of a row that a wave takes

// Values of one vector as floats: the table's own, or RN(q s).
template <class T, int N>
struct TableRow {
  const T* at;
  RawRow<T, N> v[4];
  __device__ __forceinline__ void load(int u, int c, int cols) { v[u].load(at, c, cols); }
  __device__ __forceinline__ float get(int u, int e) const { return v[u][e]; }
};
template <int N>
struct CodeRow {
  const int8_t* at;
  float s;
  CodeWords<N> v[4];
  __device__ __forceinline__ void load(int u, int c, int cols) { v[u].load(at, c, cols); }
  __device__ __forceinline__ float get(int u, int e) const { return mul_rn(v[u][e], s); }
};

template <class T, bool CODES>
__global__ void __launch_bounds__(256) embedding_kernel(const EmbedArgs p) {
  constexpr int N = kVec<T>;
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + p.first;
  const int64_t row = p.chunks == 1 ? unit : unit / p.chunks;
  if (row >= p.rows) return;
  const int c0 = (int)(unit - row * p.chunks) * kWaveVectors * N + lane * N;
  const int cols = (int)p.cols;
  const int64_t t = uniform64(p.tokens[row]);
  const bool token = t >= 0 && t < p.vocab;
  T* y = static_cast<T*>(p.Y) + row * p.ldy;
  if (!token) {
    const float zero[N] = {};
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (c0 + u * 64 * N < cols) store_row<T>(y, c0 + u * 64 * N, cols, zero);
    return;
  }
  std::conditional_t<CODES, CodeRow<N>, TableRow<T, N>> w;
  if constexpr (CODES) {
    w.at = static_cast<const int8_t*>(p.W) + t * p.ldw;
    w.s = p.scale[t];
  } else {
    w.at = static_cast<const T*>(p.W) + t * p.ldw;
  }
  const T* pos = nullptr;
  if (p.P) {
    const int64_t at = uniform64(p.positions[row]);
    if (at >= 0 && at < p.n_pos) pos = static_cast<const T*>(p.P) + at * p.ldp;
  }
  RawRow<T, N> add[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (c0 + u * 64 * N < cols) {
      w.load(u, c0 + u * 64 * N, cols);
      if (pos) add[u].load(pos, c0 + u * 64 * N, cols);
    }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (c0 + u * 64 * N < cols) {
      float v[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[e] = mul_rn(w.get(u, e), p.alpha);
        if (pos) v[e] = add_rn(v[e], add[u][e]);
      }
      store_row<T>(y, c0 + u * 64 * N, cols, v);
    }
}

// ---- the order of the tokens --------------------------------------------------------
constexpr int kRun = 8192;                     // tokens that a workgroup sorts
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kDigit = 9;                      // bits of a pass at most
constexpr int kMerge = 8;                      // runs that a merging launch joins to one

struct FillArgs {              // the rows of dW before the sums: zeros, or those of `add`
  float* dW;
  int64_t lddw, vocab, cols;
  const float* add;            // null: zeros
  int64_t ldadd;
  int blocks;                  // workgroups that fill; 0 where dW is `add`
};
struct SortArgs {
  const int64_t* tokens;
  int64_t rows, vocab;
  int bits;                    // of the keys 0 ... vocab (vocab: no token)
  uint32_t *keys, *order;      // [rows]: sorted within each run of kRun
  int runs;
};

__device__ __forceinline__ void fill_rows(const FillArgs& p, int block) {
  // whole rows a wave; 4 vectors of 4 values a lane in flight
  const int lane = threadIdx.x & 63, wave = block * kSortWaves + (threadIdx.x >> 6), waves = p.blocks * kSortWaves;
  const int cols = (int)p.cols;
  for (int64_t v = wave; v < p.vocab; v += waves) {
    float* to = p.dW + v * p.lddw;
    const float* from = p.add ? p.add + v * p.ldadd : nullptr;
    for (int c = lane * 4; c < cols; c += 256) {
      float x[4] = {};
      if (from) load_row<float, 4>(from, c, cols, 0.0f, x);
      store_row<float>(to, c, cols, x);
    }
  }
}

__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(const SortArgs p, const FillArgs fill) {
  if ((int)blockIdx.x >= p.runs) {
    fill_rows(fill, (int)blockIdx.x - p.runs);
    return;
  }
  __shared__ uint32_t key[2][kRun];
  __shared__ uint16_t at[2][kRun];
  __shared__ uint32_t count[(1 << kDigit) * kSortWaves];   // [digit][wave]
  __shared__ uint32_t wave_sum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t first = (int64_t)blockIdx.x * kRun;
  const int n = (int)min((int64_t)kRun, p.rows - first);
  for (int i = tid; i < n; i += kSortThreads) {
    const int64_t t = p.tokens[first + i];
    key[0][i] = t >= 0 && t < p.vocab ? (uint32_t)t : (uint32_t)p.vocab;
    at[0][i] = (uint16_t)i;
  }
  const int passes = (p.bits + kDigit - 1) / kDigit, width = (p.bits + passes - 1) / passes, bins = 1 << width;
  // a wave's keys: kRun / kSortWaves in a row, or what an even share of fewer is
  const int share = (n + kSortThreads - 1) / kSortThreads * 64;
  const int begin = min(wave * share, n), end = min(begin + share, n);
  int from = 0;
  for (int pass = 0; pass < passes; ++pass, from ^= 1) {
    const int shift = pass * width;
    for (int i = tid; i < bins * kSortWaves; i += kSortThreads) count[i] = 0;
    __syncthreads();
    for (int i = begin + lane; i < end; i += 64)
      atomicAdd(&count[((key[from][i] >> shift) & (bins - 1)) * kSortWaves + wave], 1u);
    __syncthreads();
    // places before each digit's and wave's keys: per consecutive counters a thread
    const int per = bins * kSortWaves / kSortThreads > 0 ? bins * kSortWaves / kSortThreads : 1;
    uint32_t mine = 0;
    if (tid * per < bins * kSortWaves)
      for (int i = 0; i < per; ++i) mine += count[tid * per + i];
    uint32_t before = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(before, d, 64);
      if (lane >= d) before += o;
    }
    if (lane == 63) wave_sum[wave] = before;
    __syncthreads();
    uint32_t base = before - mine;
    for (int w = 0; w < wave; ++w) base += wave_sum[w];
    if (tid * per < bins * kSortWaves)
      for (int i = 0; i < per; ++i) {
        const uint32_t c = count[tid * per + i];
        count[tid * per + i] = base;
        base += c;
      }
    __syncthreads();
    for (int i0 = begin; i0 < end; i0 += 64) {
      const int i = i0 + lane;
      const bool here = i < end;
      const uint32_t k = here ? key[from][i] : 0;
      const uint32_t digit = (k >> shift) & (bins - 1);
      uint64_t same = __builtin_amdgcn_ballot_w64(here);
      for (int b = 0; b < width; ++b) {
        const uint64_t m = __builtin_amdgcn_ballot_w64((digit >> b) & 1);
        same &= (digit >> b) & 1 ? m : ~m;
      }
      if (here) {
        uint32_t* c = &count[digit * kSortWaves + wave];
        const uint32_t lower = __popcll(same & ((1ull << lane) - 1));
        const uint32_t to = *c + lower;
        key[from ^ 1][to] = k;
        at[from ^ 1][to] = at[from][i];
        // the last of the digit's lanes moves the wave's place on (every lane
        // has read it: one wave's LDS accesses are in order)
        if ((same >> lane) == 1) *c = to + 1;
      }
    }
    __syncthreads();
  }
  for (int i = tid; i < n; i += kSortThreads) {
    p.keys[first + i] = key[from][i];
    p.order[first + i] = (uint32_t)(first + at[from][i]);
  }
}

// kMerge sorted runs of `run` places each to one: an element's place is its own
// plus, for each other run of its group, the elements there that come before
// it (equal ones of earlier runs do).
struct MergeArgs {
  const uint32_t *keys, *order;
  uint32_t *keys_out, *order_out;
  int64_t rows, run;
};
__global__ void __launch_bounds__(256) embedding_merge_kernel(const MergeArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.rows) return;
  const uint32_t k = p.keys[i];
  const int64_t own = i / p.run, group = own / kMerge * kMerge;
  int64_t place = group * p.run + (i - own * p.run);
  for (int64_t r = group; r < group + kMerge; ++r) {
    const int64_t start = r * p.run;
    if (r == own || start >= p.rows) continue;
    const uint32_t* a = p.keys + start;
    int64_t lo = 0, hi = min(p.run, p.rows - start);
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (a[mid] < k || (r < own && a[mid] == k)) lo = mid + 1;
      else hi = mid;
    }
    place += lo;
  }
  p.keys_out[place] = k;
  p.order_out[place] = p.order[i];
}

// ---- the sums -----------------------------------------------------------------------
constexpr int kPiece = 16;                     // places of the order that a wave takes
constexpr int kAhead = 8;                      // rows in flight

struct SumArgs {
  const void* dY;
  int64_t rows, cols, lddy, vocab;
  const uint32_t *keys, *order;
  double alpha;
  float* dW;
  int64_t lddw;
  int onto;                    // dW holds what the sums are added to
  double* parts;               // [pieces][2][cols]: sums of the piece's part of a token that began before it, and
                               // of one that goes on behind it
  int64_t pieces;
  int chunks;                  // of 64 vectors
  int64_t first;               // unit
};

template <int N>
__device__ __forceinline__ void write_row(const SumArgs& p, uint32_t token, int c, const double (&s)[N]) {
  float* to = p.dW + (int64_t)token * p.lddw;
  const int cols = (int)p.cols;
  float o[N], y[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = 0.0f;
  if (p.onto) load_row<float, N>(to, c, cols, 0.0f, o);
#pragma unroll
  for (int e = 0; e < N; ++e) y[e] = (float)(p.onto ? (double)o[e] + p.alpha * s[e] : p.alpha * s[e]);
#pragma unroll
  for (int h = 0; h < N / 4; ++h) {
    const float q[4] = {y[4 * h], y[4 * h + 1], y[4 * h + 2], y[4 * h + 3]};
    if (c + 4 * h < cols) store_row<float>(to, c + 4 * h, cols, q);
  }
}
template <int N>
__device__ __forceinline__ void leave_part(const SumArgs& p, int64_t piece, int which, int c, const double (&s)[N]) {
  double* to = p.parts + (piece * 2 + which) * p.cols;
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (c + e < (int)p.cols) to[c + e] = s[e];
}

// WHOLE: every lane's vector lies in the row (loads without a condition stay
// where they are written, ahead of their use).
template <class T, bool WHOLE>
__device__ __forceinline__ void sum_piece(const SumArgs& p, int64_t piece, int c) {
  constexpr int N = kVec<T>;
  const int lane = threadIdx.x & 63;
  const int cols = (int)p.cols;
  const int64_t begin = piece * kPiece, end = min(begin + kPiece, p.rows);
  if (uniform(p.keys[begin]) >= (uint32_t)p.vocab) return;         // what is no token sorts last
  const bool went_on = begin > 0 && uniform(p.keys[begin - 1]) == uniform(p.keys[begin]);
  const bool goes_on = end < p.rows && uniform(p.keys[end]) == uniform(p.keys[end - 1]);
  // the places' tokens and rows, one a lane
  const int n = (int)(end - begin);
  const uint32_t my_key = lane < n ? p.keys[begin + lane] : 0xFFFFFFFFu;
  const uint32_t my_row = p.order[begin + min(lane, n - 1)];
  const T* dy = static_cast<const T*>(p.dY);
  RawRow<T, N> ahead[kAhead];
  auto load = [&](int i) {
    const T* row = dy + (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)my_row, i) * p.lddy;
    if constexpr (WHOLE) __builtin_memcpy(ahead[i % kAhead].t, row + c, sizeof(ahead[0].t));
    else ahead[i % kAhead].load(row, c, cols);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i);
  double s[N];
#pragma unroll
  for (int e = 0; e < N; ++e) s[e] = 0.0;
  bool head = went_on;
#pragma unroll
  for (int i = 0; i < kPiece; ++i) {
    if (i >= n) break;
    const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)my_key, i);
    if (key >= (uint32_t)p.vocab) break;
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] += (double)ahead[i % kAhead][e];
    if (i + kAhead < kPiece) load(i + kAhead);
    const bool last = i + 1 == n;
    if (last || (uint32_t)__builtin_amdgcn_readlane((int)my_key, i + 1) != key) {
      if (WHOLE || c < cols) {
        if (head) leave_part<N>(p, piece, 0, c, s);
        else if (last && goes_on) leave_part<N>(p, piece, 1, c, s);
        else write_row<N>(p, key, c, s);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) s[e] = 0.0;
      head = false;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(256) embedding_sum_kernel(const SumArgs p) {
  constexpr int N = kVec<T>;
  const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + p.first;
  const int64_t piece = p.chunks == 1 ? unit : unit / p.chunks;
  if (piece >= p.pieces) return;
  const int c0 = (int)(unit - piece * p.chunks) * 64 * N;
  const int c = c0 + (threadIdx.x & 63) * N;
  if (c0 + 64 * N <= (int)p.cols) sum_piece<T, true>(p, piece, c);
  else sum_piece<T, false>(p, piece, c);
}

// A workgroup for each piece and 64 columns: where a token's places begin in
// the piece and go on behind it, its parts are added, 4 waves taking every
// fourth, the waves' sums in their order.
__global__ void __launch_bounds__(256) embedding_join_kernel(const SumArgs p) {
  const int64_t unit = (int64_t)blockIdx.x + p.first;
  const int64_t piece = unit / p.chunks;
  const int64_t end = (piece + 1) * kPiece;
  if (end >= p.rows) return;
  const uint32_t key = uniform(p.keys[end - 1]);
  if (uniform(p.keys[end]) != key || key >= (uint32_t)p.vocab) return;
  const int64_t begin = piece * kPiece;
  if (uniform(p.keys[begin]) == key && begin > 0 && uniform(p.keys[begin - 1]) == key) return;   // began earlier
  // the last place of the token
  int64_t lo = end, hi = p.rows;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (uniform(p.keys[mid]) == key) lo = mid + 1;
    else hi = mid;
  }
  const int64_t last = (lo - 1) / kPiece;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (int)(unit - piece * p.chunks) * 64 + lane;
  const bool in = c < (int)p.cols;
  double s = 0.0;
  if (in) {
    if (wave == 0) s = p.parts[(piece * 2 + 1) * p.cols + c];
#pragma unroll 4
    for (int64_t q = piece + 1 + wave; q <= last; q += 4) s += p.parts[q * 2 * p.cols + c];
  }
  __shared__ double sum[4][64];
  sum[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || !in) return;
  s = (sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]);
  float* to = p.dW + (int64_t)key * p.lddw + c;
  *to = (float)(p.onto ? (double)*to + p.alpha * s : p.alpha * s);
}

// Launches of at most 2^22 workgroups.
template <class Launch>
hipError_t in_slabs(int64_t blocks, Launch launch) {
  constexpr int64_t most = int64_t(1) << 22;
  for (int64_t b = 0; b < blocks; b += most) {
    launch((unsigned)(blocks - b < most ? blocks - b : most), b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
int64_t up64(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t aligned(size_t n) { return (n + 255) / 256 * 256; }
int64_t merges(int64_t rows) {
  int64_t n = 0;
  for (int64_t run = kRun; run < rows; run *= kMerge) ++n;
  return n;
}

}  // namespace

hipError_t launch_embedding(EmbedArgs a, int dtype, bool codes, hipStream_t stream) {
  const int n = dtype == DT_F32 ? 4 : 8;
  a.chunks = (int)up64(a.cols, (int64_t)kWaveVectors * n);
  return in_slabs(up64(a.rows * a.chunks, 4), [&](unsigned grid, int64_t first) {
    a.first = first * 4;
    const dim3 g(grid), b(256);
    if (dtype == DT_F32 && codes) hipLaunchKernelGGL((embedding_kernel<float, true>), g, b, 0, stream, a);
    else if (dtype == DT_BF16 && codes) hipLaunchKernelGGL((embedding_kernel<bf16_t, true>), g, b, 0, stream, a);
    else if (codes) hipLaunchKernelGGL((embedding_kernel<f16_t, true>), g, b, 0, stream, a);
    else if (dtype == DT_F32) hipLaunchKernelGGL((embedding_kernel<float, false>), g, b, 0, stream, a);
    else if (dtype == DT_BF16) hipLaunchKernelGGL((embedding_kernel<bf16_t, false>), g, b, 0, stream, a);
    else hipLaunchKernelGGL((embedding_kernel<f16_t, false>), g, b, 0, stream, a);
  });
}

// The workspace: the sorted keys and rows (twice where runs are merged), then
// the parts.
size_t embedding_bwd_bytes(int64_t rows, int64_t cols) {
  const size_t list = aligned((size_t)rows * 4);
  return list * (merges(rows) > 0 ? 4 : 2) + aligned((size_t)up64(rows, kPiece) * 2 * (size_t)cols * 8);
}

hipError_t launch_embedding_bwd(const EmbedBwdArgs& a, int dtype, void* ws, hipStream_t stream) {
  char* at = static_cast<char*>(ws);
  const size_t list = aligned((size_t)a.rows * 4);
  const int64_t n_merges = merges(a.rows);
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(at), reinterpret_cast<uint32_t*>(at + 2 * list)};
  uint32_t* order[2] = {reinterpret_cast<uint32_t*>(at + list), reinterpret_cast<uint32_t*>(at + 3 * list)};
  double* parts = reinterpret_cast<double*>(at + list * (n_merges > 0 ? 4 : 2));
  const bool in_place = a.add == a.dW;
  SortArgs s{a.tokens, a.rows, a.vocab, 0, keys[0], order[0], (int)up64(a.rows, kRun)};
  while ((a.vocab >> s.bits) != 0) ++s.bits;              // vocab itself is a key
  if (s.bits == 0) s.bits = 1;
  // 1024 workgroups fill: 4 for each of the 256 CUs
  FillArgs f{a.dW, a.lddw, a.vocab, a.cols, a.add, a.ldadd, in_place ? 0 : (int)(up64(a.vocab, kSortWaves) < 1024 ? up64(a.vocab, kSortWaves) : 1024)};
  if (s.runs + f.blocks > 0) hipLaunchKernelGGL(embedding_sort_kernel, dim3((unsigned)(s.runs + f.blocks)), dim3(kSortThreads), 0, stream, s, f);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.rows == 0) return e;
  int from = 0;
  for (int64_t run = kRun; run < a.rows; run *= kMerge, from ^= 1) {
    MergeArgs m{keys[from], order[from], keys[from ^ 1], order[from ^ 1], a.rows, run};
    hipLaunchKernelGGL(embedding_merge_kernel, dim3((unsigned)up64(a.rows, 256)), dim3(256), 0, stream, m);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const int n = dtype == DT_F32 ? 4 : 8;
  SumArgs u{a.dY, a.rows, a.cols, a.lddy, a.vocab, keys[from], order[from], (double)a.alpha, a.dW, a.lddw, a.add != nullptr,
            parts, up64(a.rows, kPiece), (int)up64(a.cols, 64 * n), 0};
  e = in_slabs(up64(u.pieces * u.chunks, 4), [&](unsigned grid, int64_t first) {
    u.first = first * 4;
    if (dtype == DT_F32) hipLaunchKernelGGL(embedding_sum_kernel<float>, dim3(grid), dim3(256), 0, stream, u);
    else if (dtype == DT_BF16) hipLaunchKernelGGL(embedding_sum_kernel<bf16_t>, dim3(grid), dim3(256), 0, stream, u);
    else hipLaunchKernelGGL(embedding_sum_kernel<f16_t>, dim3(grid), dim3(256), 0, stream, u);
  });
  if (e != hipSuccess || u.pieces == 1) return e;
  u.chunks = (int)up64(a.cols, 64);
  return in_slabs((u.pieces - 1) * u.chunks, [&](unsigned grid, int64_t first) {
    u.first = first;
    hipLaunchKernelGGL(embedding_join_kernel, dim3(grid), dim3(256), 0, stream, u);
  });
}

}  // namespace i8g
