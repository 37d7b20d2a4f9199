// embedding.hip -- rows of a table looked up by token, and the table's
// gradient.
//
//   Y_i  = RN(alpha W[t_i]) + P[p_i]         W in f32, bf16, f16, or codes and scales: W = RN(q s)
//   dW_v = alpha sum_{t_i = v} dY_i          binary64 sums
//
// The lookup is one pass: a wave takes up to 256 vectors of a row, four loads
// in flight.  The gradient of few rows is one launch that looks through all
// tokens.  That of more sorts them, while other workgroups fill dW with zeros or
// with what is added to (up to kRankRows each key's place is counted by the whole
// chip; beyond, a stable radix sort of kRun at a time in LDS, the sorted runs
// merged kMerge at a time), then adds rows in the sorted order: a wave takes a
// piece of the order and a chunk of columns, writes the rows of tokens whose
// places it holds all of, and leaves the others' sums in the workspace, which
// a last launch joins.  What is added to what follows from the sizes and the
// tokens alone: four sums, of every fourth 64 rows each, where all tokens are looked
// through, else the pieces' sums, each in the order of i; and no sum depends on which
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

// Memory: 8192 x 768 f32 with positions 9.4 us, 5.7 TB/s; from codes into bf16 7.7
// us for 20 MB, where the token's load, then the row's, then the store are most of
// a wave's time.
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
  int lanes_log;
  int64_t first, end;          // rows of the launch
  int blocks;                  // workgroups that fill; 0 where dW is `add`
};
// The pieces that left a second sum (see the sums) are listed by a counter each
// kLists-th piece has: 4 kB of them, 64 bytes apart, so that two share one of the
// L2's lines of 128.  (On one address the additions take some 10 ns each, one after
// the other: 32000 x 76 took 22 us, and 6.4 with these.)
constexpr int kLists = 64, kListStep = 16;
__device__ __forceinline__ void clear_lists(uint32_t* listed) {
  if (threadIdx.x < kLists) listed[threadIdx.x * kListStep] = 0;
}

struct SortArgs {
  const int64_t* tokens;
  int64_t rows, vocab;
  int bits;                    // of the keys 0 ... vocab (vocab: no token)
  uint32_t *keys, *order;      // [rows]: sorted within each run of kRun
  int runs;
  uint32_t* listed;            // the lists' counters, zeroed for the sums
};

// Rows v0 ... of a wave, as many as 64 lanes hold at 4 columns each (all lanes one
// row of 256 columns or more): lane l has row v0 + (l >> lanes_log).
int lanes_log(int64_t cols) {
  int n = 0;
  while (n < 6 && (int64_t(4) << n) < cols) ++n;
  return n;
}
__device__ __forceinline__ void fill_row(const FillArgs& p, int64_t v) {
  const int in = threadIdx.x & ((1 << p.lanes_log) - 1), step = 4 << p.lanes_log;
  const int cols = (int)p.cols;
  float* to = p.dW + v * p.lddw;
  const float* from = p.add ? p.add + v * p.ldadd : nullptr;
  for (int c = in * 4; c < cols; c += step) {
    float x[4] = {};
    if (from) load_row<float, 4>(from, c, cols, 0.0f, x);
    stream_row<float>(to, c, cols, x);
  }
}
template <int WAVES>
__device__ __forceinline__ void fill_rows(const FillArgs& p, int block) {
  const int rows = 64 >> p.lanes_log, lane_row = (threadIdx.x & 63) >> p.lanes_log;
  const int64_t wave = block * WAVES + (threadIdx.x >> 6), waves = p.blocks * WAVES;
  for (int64_t v = p.first + wave * rows + lane_row; v < p.end; v += waves * rows) fill_row(p, v);
}

// A stable radix sort of up to kRun tokens a workgroup, kDigit bits a pass: a wave
// counts its keys' digits, and the lanes of a digit find their places by ballots.
// 8192 tokens of 14 bits 20 us, all of it LDS latency in 16 waves, so the table's
// rows are written beside it: 247 MB read or written in 47 us, 5.3 TB/s.
__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(const SortArgs p, const FillArgs fill) {
  if ((int)blockIdx.x >= p.runs) {
    fill_rows<kSortWaves>(fill, (int)blockIdx.x - p.runs);
    return;
  }
  if (blockIdx.x == 0) clear_lists(p.listed);
  __shared__ uint32_t key[2][kRun];
  __shared__ uint16_t at[2][kRun];
  __shared__ uint32_t count[(1 << kDigit) * kSortWaves];   // [digit][wave]
  __shared__ uint32_t wave_sum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t first = (int64_t)blockIdx.x * kRun;
  const int n = (int)min((int64_t)kRun, p.rows - first);
  constexpr int kOwn = kRun / kSortThreads;
  int64_t t[kOwn];
#pragma unroll
  for (int q = 0; q < kOwn; ++q) t[q] = p.tokens[first + min(tid + q * kSortThreads, n - 1)];
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    const int i = tid + q * kSortThreads;
    if (i < n) {
      key[0][i] = t[q] >= 0 && t[q] < p.vocab ? (uint32_t)t[q] : (uint32_t)p.vocab;
      at[0][i] = (uint16_t)i;
    }
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

// Few enough rows are sorted by the whole chip: a workgroup has all keys in LDS
// and finds the places of kRank of them, as the keys that come before each: a
// thread counts for one row over an even share of them.  (With the table hardly
// larger than the tokens, 3363 rows take 8 us and 8192 14, and 12 and 21 where a
// workgroup sorts up to kRun of them; 11270 24 and 33, with the merge; 16384 34
// and 33.)
constexpr int kRank = 32, kRankThreads = 512, kRankRows = 12288;
constexpr int kRankShares = kRankThreads / kRank;
static_assert(kRank == 32, "the loops below");
__global__ void __launch_bounds__(kRankThreads) embedding_rank_kernel(const SortArgs p, const FillArgs fill) {
  if ((int)blockIdx.x >= p.runs) {
    fill_rows<kRankThreads / 64>(fill, (int)blockIdx.x - p.runs);
    return;
  }
  if (blockIdx.x == 0) clear_lists(p.listed);
  extern __shared__ __attribute__((aligned(16))) uint32_t keys[];          // whole kRanks, those behind the rows 2^32 - 1
  __shared__ uint32_t count[kRankThreads / 64][kRank];
  const int tid = threadIdx.x, rows = (int)p.rows, all = (rows + kRank - 1) / kRank * kRank;
  for (int i0 = tid; i0 < all; i0 += 8 * kRankThreads) {
    int64_t t[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) t[q] = p.tokens[min(i0 + q * kRankThreads, rows - 1)];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int i = i0 + q * kRankThreads;
      if (i < all) keys[i] = i >= rows ? 0xFFFFFFFFu : t[q] >= 0 && t[q] < p.vocab ? (uint32_t)t[q] : (uint32_t)p.vocab;
    }
  }
  __syncthreads();
  const int first = (int)blockIdx.x * kRank, own = first + tid % kRank, share = tid / kRank;
  const int per = (all / kRank + kRankShares - 1) / kRankShares * kRank;   // keys of a share
  const int begin = min(share * per, all), end = min(begin + per, all);
  const uint32_t mine = keys[own];
  uint32_t n = 0;
  const auto below = [&](int from, int to, uint32_t limit) {
    for (int i = from; i < to; i += 32) {                  // (all are whole kRanks)
      uint4 k[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) k[q] = *reinterpret_cast<const uint4*>(keys + i + 4 * q);
#pragma unroll
      for (int q = 0; q < 8; ++q) n += (k[q].x < limit) + (k[q].y < limit) + (k[q].z < limit) + (k[q].w < limit);
    }
  };
  below(begin, min(end, first), mine + 1);                 // equal ones of earlier rows come before it
  below(max(begin, first + kRank), end, mine);
#pragma unroll
  for (int i = share * (kRank / kRankShares); i < (share + 1) * (kRank / kRankShares); ++i) {
    const uint32_t k = keys[first + i];
    n += k < mine || (k == mine && first + i < own);
  }
  n += __shfl_xor(n, 32, 64);
  if ((tid & 63) < kRank) count[tid >> 6][tid & 63] = n;
  __syncthreads();
  if (tid >= kRank || own >= rows) return;
  uint32_t place = 0;
#pragma unroll
  for (int w = 0; w < kRankThreads / 64; ++w) place += count[w][tid];
  p.keys[place] = mine;
  p.order[place] = (uint32_t)own;
}

// kMerge sorted runs of `run` places each to one: an element's place is its own
// plus, for each other run of its group, the elements there that come before
// it (equal ones of earlier runs do).  42851 places 13 us, the latency of 14 steps
// of search.
struct MergeArgs {
  const uint32_t *keys, *order;
  uint32_t *keys_out, *order_out;
  int64_t rows, run;
  int64_t groups;              // workgroups that merge; those behind fill
};
__global__ void __launch_bounds__(256) embedding_merge_kernel(const MergeArgs p, const FillArgs fill) {
  if (blockIdx.x >= p.groups) {
    fill_rows<4>(fill, (int)(blockIdx.x - p.groups));
    return;
  }
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.rows) return;
  const uint32_t k = p.keys[i];
  const int64_t own = i / p.run, group = own / kMerge * kMerge;
  int64_t place = i - (own - group) * p.run;
  // the searches side by side: each step's loads are independent
  int64_t before[kMerge];
#pragma unroll
  for (int r = 0; r < kMerge; ++r) before[r] = 0;
  for (int64_t step = p.run; step > 0; step >>= 1) {
    uint32_t a[kMerge];
#pragma unroll
    for (int r = 0; r < kMerge; ++r) a[r] = p.keys[min((group + r) * p.run + before[r] + step, p.rows) - 1];
#pragma unroll
    for (int r = 0; r < kMerge; ++r) {
      const int64_t at = before[r] + step;       // are the run's first `at` before it?
      const bool there = group + r != own && at <= p.run && (group + r) * p.run + at <= p.rows;
      if (there && (a[r] < k || (a[r] == k && group + r < own))) before[r] = at;
    }
  }
#pragma unroll
  for (int r = 0; r < kMerge; ++r) place += before[r];
  p.keys_out[place] = k;
  p.order_out[place] = p.order[i];
}

// ---- few rows: one launch ------------------------------------------------------------
// Every wave holds all tokens, WORDS a lane.  The workgroups of a row take 256
// columns at a time: if no earlier row has its token, they add all that have, each
// wave those of every fourth 64 rows, the waves' sums in their order.  The
// workgroups behind fill the rows of the table that no token names.  Against the
// three launches of sorting, adding and joining (us): 64 x 768 onto 100 rows 4.1
// and 11.0, 256 x 5000 onto 300 10.4 and 17.7, 700 x 76 onto 31438 14.4 and 17.7,
// 1024 x 768 onto 1024 13.5 and 15.8; but 512 x 4096 onto 1024 19.7 and 15.0,
// 918 x 2252 onto 1365 24 and 19, as every workgroup looks through all tokens.
constexpr int kFewWords = 16, kFew = kFewWords * 64, kFewGroups = 2048;
bool few_rows(int64_t rows, int64_t cols) {
  return rows <= 256 || (rows <= kFew && rows * ((cols + 255) / 256) <= 3 * kFew);
}
struct FewArgs {
  const void* dY;
  int64_t rows, cols, lddy;
  const int64_t* tokens;
  double alpha;
  int chunks;                  // workgroups of a row
  int64_t sums;                // workgroups that add
  FillArgs fill;
};
// WHOLE: as for the sums below.
template <class T, int WORDS, bool WHOLE>
__device__ __forceinline__ void few_sums(const FewArgs& p, const uint64_t (&has)[WORDS], double (&sum)[4][64][4], int64_t token,
                                         int c, int wave) {
  constexpr int N = 4;
  const int lane = threadIdx.x & 63, cols = (int)p.cols;
  double s[N];
#pragma unroll
  for (int e = 0; e < N; ++e) s[e] = 0.0;
#pragma unroll
  for (int w = 0; w < WORDS; w += 4) {
    uint64_t mine = wave == 0 ? has[w] : wave == 1 ? has[w + 1] : wave == 2 ? has[w + 2] : has[w + 3];
    const T* dy = static_cast<const T*>(p.dY) + (int64_t)((w + wave) * 64) * p.lddy;
    while (mine != 0) {
      RawRow<T, N> x[8];
      uint64_t left = mine;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = __builtin_ctzll(left != 0 ? left : mine);
        left &= left - 1;
        if constexpr (WHOLE) __builtin_memcpy(x[i].t, dy + at * p.lddy + c, sizeof(x[i].t));
        else x[i].load(dy + at * p.lddy, c, cols);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (mine != 0) {
#pragma unroll
          for (int e = 0; e < N; ++e) s[e] += (double)x[i][e];
          mine &= mine - 1;
        }
    }
  }
#pragma unroll
  for (int e = 0; e < N; ++e) sum[wave][lane][e] = s[e];
  __syncthreads();
  if (wave != 0 || (!WHOLE && c >= cols)) return;
  float y[N], old[N];
  if (p.fill.add) load_row<float, N>(p.fill.add + token * p.fill.ldadd, c, cols, 0.0f, old);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const double all = p.alpha * (((sum[0][lane][e] + sum[1][lane][e]) + sum[2][lane][e]) + sum[3][lane][e]);
    y[e] = (float)(p.fill.add ? (double)old[e] + all : all);
  }
  store_row<float, N>(p.fill.dW + token * p.fill.lddw, c, cols, y);
}

template <class T, int WORDS>
__global__ void __launch_bounds__(256) embedding_few_kernel(const FewArgs p) {
  constexpr int N = 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = (int)p.cols;
  int t[WORDS];                                  // (at most 2^31 - 1; -1: no token)
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    const int64_t x = p.tokens[min(w * 64 + lane, (int)p.rows - 1)];
    t[w] = w * 64 + lane < (int)p.rows && x >= 0 && x < p.fill.vocab ? (int)x : -1;
  }
  if (blockIdx.x >= p.sums) {
    const FillArgs& f = p.fill;
    const int rows = 64 >> f.lanes_log, lane_row = lane >> f.lanes_log;
    const int64_t waves = (int64_t)(gridDim.x - p.sums) * 4;
    for (int64_t v0 = ((int64_t)(blockIdx.x - p.sums) * 4 + wave) * rows; v0 < f.vocab; v0 += waves * rows) {
      uint64_t named = 0;                        // of the wave's rows
      for (int r = 0; r < rows; ++r) {
        bool here = false;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) here = here || t[w] == (int)(v0 + r);
        if (__builtin_amdgcn_ballot_w64(here) != 0) named |= 1ull << r;
      }
      if (v0 + lane_row < f.vocab && ((named >> lane_row) & 1) == 0) fill_row(f, v0 + lane_row);
    }
    return;
  }
  const int row = (int)(p.chunks == 1 ? blockIdx.x : blockIdx.x / p.chunks);
  const int chunk = (int)(blockIdx.x - (int64_t)row * p.chunks);
  const int64_t token = uniform64(p.tokens[row]);
  if (token < 0 || token >= p.fill.vocab) return;
  bool earlier = false;
  uint64_t has[WORDS];
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    has[w] = __builtin_amdgcn_ballot_w64(t[w] == (int)token);
    if (w < (row >> 6)) earlier = earlier || has[w] != 0;
    if (w == (row >> 6)) earlier = earlier || (has[w] & ((1ull << (row & 63)) - 1)) != 0;
  }
  if (earlier) return;
  __shared__ double sum[4][64][N];
  for (int64_t first = (int64_t)chunk * 64 * N; first < cols; first += (int64_t)p.chunks * 64 * N) {
    const int c = (int)first + lane * N;
    if (cols - (int)first >= N) few_sums<T, WORDS, true>(p, has, sum, token, min(c, cols - N), wave);
    else few_sums<T, WORDS, false>(p, has, sum, token, c, wave);
    __syncthreads();
  }
}
template <int WORDS>
void launch_few(int dtype, dim3 grid, hipStream_t stream, const FewArgs& a) {
  if (dtype == DT_F32) hipLaunchKernelGGL((embedding_few_kernel<float, WORDS>), grid, dim3(256), 0, stream, a);
  else if (dtype == DT_BF16) hipLaunchKernelGGL((embedding_few_kernel<bf16_t, WORDS>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((embedding_few_kernel<f16_t, WORDS>), grid, dim3(256), 0, stream, a);
}

// ---- the sums -----------------------------------------------------------------------
constexpr int kLane = 4;                       // columns of a lane
// Places whose rows a wave has in flight (fewer where the rows that they are
// added to are, too).
template <bool ONTO>
constexpr int kBatch = ONTO ? 8 : 16;
constexpr int kPlaces = 16;                    // a piece is a multiple of

struct SumArgs {
  const void* dY;
  int64_t rows, cols, lddy, vocab;
  const uint32_t *keys, *order;
  double alpha;
  float* dW;
  int64_t lddw;
  int onto;                    // dW holds what the sums are added to
  int64_t piece, pieces;       // places of a piece (a multiple of kBatch), and how many there are
  double* parts;               // [pieces][2][ldp]: sums of the piece's part of a token that began before it, and
                               // of one that goes on behind it
  int64_t ldp;                 // cols in whole chunks
  uint32_t *list, *listed;     // the pieces that left a second sum: kLists lists, and how many are in each
  int64_t list_ld;
  int chunks;                  // of 64 vectors
  int64_t first;               // unit
};

template <int B, int E, class F>
__device__ __forceinline__ void for_each(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    for_each<B + 1, E>(f);
  }
}

// WHOLE: every lane's columns lie in the row, where the last lanes' begin before
// theirs so that they do: these have what others have too, to the bit.  (Loads
// without a condition stay where they are written, ahead of their use: 2135 x 207
// takes 5.6 us, and 9.3 with conditions.)
template <class T, bool WHOLE, bool ONTO>
__device__ __forceinline__ void sum_piece(const SumArgs& p, int64_t piece, int c, bool first) {
  constexpr int N = kLane, B = kBatch<ONTO>;
  const int lane = threadIdx.x & 63;
  const int cols = (int)p.cols;
  const int64_t begin = piece * p.piece, end = min(begin + p.piece, p.rows);
  const uint32_t vocab = (uint32_t)p.vocab;
  bool head = false;                             // the sum began before the piece
  const T* dy = static_cast<const T*>(p.dY);
  double* parts = p.parts + piece * 2 * p.ldp + c;
  double s[N];
#pragma unroll
  for (int e = 0; e < N; ++e) s[e] = 0.0;
  for (int64_t at = begin; at < end; at += B) {
    // lane i: the token and the row of place i - 1 (so the first one's is the
    // place before the batch, the last one's the place behind it)
    const int64_t mine = at - 1 + min(lane, B + 1);
    const uint32_t my_key = mine >= 0 && mine < p.rows ? p.keys[mine] : 0xFFFFFFFFu;
    const uint32_t my_row = p.order[min(max(mine, begin), end - 1)];
    const int places = (int)min((int64_t)B, end - at);
    const int n = __popcll(__builtin_amdgcn_ballot_w64(lane >= 1 && lane <= places && my_key < vocab));   // (no token sorts last)
    if (at == begin) head = __builtin_amdgcn_readlane((int)my_key, 0) == __builtin_amdgcn_readlane((int)my_key, 1);
    if (n == 0) return;
    RawRow<T, N> row[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const T* r = dy + (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)my_row, i + 1) * p.lddy;
      if constexpr (WHOLE) __builtin_memcpy(row[i].t, r + c, sizeof(row[i].t));
      else row[i].load(r, c, cols);
    }
    // the rows that sums of this batch are added to
    RawRow<float, N> old[B];
    if constexpr (ONTO) {
      for_each<0, B>([&](auto i) {
        const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)my_key, i + 1);
        if (i < n && (uint32_t)__builtin_amdgcn_readlane((int)my_key, i + 2) != key) {
          const float* from = p.dW + (int64_t)key * p.lddw;
          if constexpr (WHOLE) __builtin_memcpy(old[i].t, from + c, sizeof(old[i].t));
          else old[i].load(from, c, cols);
        }
      });
    }
    for_each<0, B>([&](auto i) {
      if (i < n) {
        const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)my_key, i + 1);
        const bool ends = (uint32_t)__builtin_amdgcn_readlane((int)my_key, i + 2) != key;
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] += (double)row[i][e];
        if (ends || at + i + 1 == end) {
          if (head || !ends) {
            __builtin_memcpy(parts + (head ? 0 : p.ldp), s, sizeof(s));
            // (a list's order is no matter: its entries have nothing in common)
            if (!head && lane == 0 && first) {
              const int l = (int)(piece % kLists);
              p.list[l * p.list_ld + atomicAdd(p.listed + l * kListStep, 1u)] = (uint32_t)piece;
            }
          } else if (WHOLE || c < cols) {
            float* to = p.dW + (int64_t)key * p.lddw;
            float y[N];
#pragma unroll
            for (int e = 0; e < N; ++e) y[e] = (float)(ONTO ? (double)old[i][e] + p.alpha * s[e] : p.alpha * s[e]);
            if constexpr (WHOLE) __builtin_memcpy(to + c, y, sizeof(y));
            else store_row<float, N>(to, c, cols, y);
          }
#pragma unroll
          for (int e = 0; e < N; ++e) s[e] = 0.0;
          head = false;
        }
      }
    });
  }
}

// A wave a piece and 256 columns.  8192 x 768 f32 8.7 us (25 MB read, at most as
// much written); 65536 x 768 bf16 added to 50257 rows 43 us: 100 MB read, and the
// rows that tokens name read and written.
template <class T, bool ONTO>
__global__ void __launch_bounds__(256) embedding_sum_kernel(const SumArgs p) {
  const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + p.first;
  const int64_t piece = p.chunks == 1 ? unit : unit / p.chunks;
  if (piece >= p.pieces) return;
  const int c0 = (int)(unit - piece * p.chunks) * 64 * kLane;
  const int c = c0 + (threadIdx.x & 63) * kLane;
  // (not into another wave's columns, which it may have added to already)
  if ((int)p.cols - c0 >= kLane) sum_piece<T, true, ONTO>(p, piece, min(c, (int)p.cols - kLane), c0 == 0);
  else sum_piece<T, false, ONTO>(p, piece, c, c0 == 0);
}

// Workgroups take a listed piece and 256 columns at a time: the sums of the
// token that goes on behind the piece, added in their order.  Latency: the list,
// the key, then the pieces that it goes on in; 4 to 9 us.
constexpr int kJoinGroups = 2048;              // whole kLists

__global__ void __launch_bounds__(256) embedding_join_kernel(const SumArgs p) {
  const int l = (int)(blockIdx.x % kLists);
  const int64_t items = (int64_t)uniform(p.listed[l * kListStep]) * p.chunks;
  for (int64_t item = blockIdx.x / kLists; item < items; item += gridDim.x / kLists) {
    const int64_t entry = p.chunks == 1 ? item : item / p.chunks;
    const int64_t piece = uniform(p.list[l * p.list_ld + entry]);
    const int64_t c = (item - entry * p.chunks) * 256 + threadIdx.x;
    const uint32_t key = uniform(p.keys[(piece + 1) * p.piece - 1]);
    // the last piece that it goes on in: 64 of their first places at a time
    int64_t last = piece + 1;
    for (;; last += 64) {
      const int64_t at = (last + 1 + (threadIdx.x & 63)) * p.piece;
      const uint64_t on = __builtin_amdgcn_ballot_w64(at < p.rows && p.keys[min(at, p.rows - 1)] == key);
      if (~on != 0) {
        last += __builtin_ctzll(~on);
        break;
      }
    }
    if (c >= p.cols) continue;
    const double* part = p.parts + c;
    double s = part[(piece * 2 + 1) * p.ldp];
    float* to = p.dW + (int64_t)key * p.lddw + c;
    const float old = p.onto ? *to : 0.0f;
    int64_t q = piece + 1;
    for (; q + 31 <= last; q += 32) {
      double x[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = part[(q + i) * 2 * p.ldp];
#pragma unroll
      for (int i = 0; i < 32; ++i) s += x[i];
    }
    for (; q <= last; q += 4) {
      double x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = part[min(q + i, last) * 2 * p.ldp];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (q + i <= last) s += x[i];
    }
    *to = (float)(p.onto ? (double)old + p.alpha * s : p.alpha * s);
  }
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

// Places of a piece: as few as leave at most about 4096 waves, 16 to 128.
int64_t piece_of(int64_t rows, int64_t cols) {
  const int64_t n = up64(rows, kPlaces) * up64(cols, 64 * kLane) / 4096;
  return kPlaces * (n < 1 ? 1 : n > 8 ? 8 : n);
}
int64_t part_ld(int64_t cols) { return up64(cols, 64 * kLane) * (64 * kLane); }

// The workspace: the sorted keys and rows (twice where runs are merged), the
// pieces to be joined and their count, and the parts.
struct BwdLayout {
  size_t list, joined, bytes;  // of a list of keys or rows; where the pieces' list and the parts begin
  size_t parts;
  int64_t list_ld;
};
BwdLayout bwd_layout(int64_t rows, int64_t cols) {
  BwdLayout l;
  const int64_t pieces = up64(rows, piece_of(rows, cols));
  l.list = aligned((size_t)rows * 4);
  l.joined = l.list * (merges(rows) > 0 ? 4 : 2);
  l.list_ld = up64(pieces, kLists);
  l.parts = l.joined + aligned((size_t)(kListStep + l.list_ld) * kLists * 4);
  l.bytes = l.parts + (size_t)pieces * 2 * (size_t)part_ld(cols) * 8;
  return l;
}
size_t embedding_bwd_bytes(int64_t rows, int64_t cols) { return bwd_layout(rows, cols).bytes; }

hipError_t launch_embedding_bwd(const EmbedBwdArgs& a, int dtype, void* ws, hipStream_t stream) {
  const bool in_place = a.add == a.dW;
  const int lanes = lanes_log(a.cols);
  const auto fill = [&](int64_t first, int64_t end, int waves) {
    const int64_t blocks = in_place ? 0 : up64(end - first, (int64_t)waves * (64 >> lanes));
    const int64_t most = 16384 / waves;                    // 4 workgroups of 16 waves for each of the 256 CUs
    return FillArgs{a.dW, a.lddw, a.vocab, a.cols, a.add, a.ldadd, lanes, first, end, (int)(blocks < most ? blocks : most)};
  };
  if (a.rows > 0 && few_rows(a.rows, a.cols)) {
    const int64_t all = up64(a.cols, 256), most = up64(kFewGroups, a.rows), chunks = all < most ? all : most;
    FewArgs w{a.dY, a.rows, a.cols, a.lddy, a.tokens, (double)a.alpha, (int)chunks, a.rows * chunks, fill(0, a.vocab, 4)};
    const dim3 grid((unsigned)(w.sums + w.fill.blocks));
    if (a.rows <= 256) launch_few<4>(dtype, grid, stream, w);
    else launch_few<kFewWords>(dtype, grid, stream, w);
    return hipGetLastError();
  }
  char* at = static_cast<char*>(ws);
  const BwdLayout lay = bwd_layout(a.rows, a.cols);
  const size_t list = lay.list;
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(at), reinterpret_cast<uint32_t*>(at + 2 * list)};
  uint32_t* order[2] = {reinterpret_cast<uint32_t*>(at + list), reinterpret_cast<uint32_t*>(at + 3 * list)};
  uint32_t* listed = reinterpret_cast<uint32_t*>(at + lay.joined);
  SortArgs s{a.tokens, a.rows, a.vocab, 0, keys[0], order[0], (int)up64(a.rows, kRun), listed};
  while ((a.vocab >> s.bits) != 0) ++s.bits;              // vocab itself is a key
  if (s.bits == 0) s.bits = 1;
  hipError_t e;
  int from = 0;
  if (a.rows > 0 && a.rows <= kRankRows) {
    s.runs = (int)up64(a.rows, kRank);
    const FillArgs f = fill(0, a.vocab, kRankThreads / 64);
    hipLaunchKernelGGL(embedding_rank_kernel, dim3((unsigned)(s.runs + f.blocks)), dim3(kRankThreads), (size_t)s.runs * kRank * 4, stream, s, f);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else {
    // The rows are filled beside the sorting and the merging, which leave most of
    // the chip free: a merge takes as long as about a fifth of a fill of 150 MB.
    int n_merges = (int)merges(a.rows);
    if (n_merges > 2) n_merges = 2;
    const int64_t later = in_place ? 0 : a.vocab / 5 * n_merges;
    FillArgs f = fill(0, a.vocab - later, kSortWaves);
    if (s.runs + f.blocks > 0) hipLaunchKernelGGL(embedding_sort_kernel, dim3((unsigned)(s.runs + f.blocks)), dim3(kSortThreads), 0, stream, s, f);
    e = hipGetLastError();
    if (e != hipSuccess || a.rows == 0) return e;
    int64_t filled = a.vocab - later;
    for (int64_t run = kRun; run < a.rows; run *= kMerge, from ^= 1) {
      MergeArgs m{keys[from], order[from], keys[from ^ 1], order[from ^ 1], a.rows, run, up64(a.rows, 256)};
      const int64_t to = run * kMerge >= a.rows ? a.vocab : filled + a.vocab / 5 < a.vocab ? filled + a.vocab / 5 : a.vocab;
      f = fill(filled, to, 4);
      filled = to;
      hipLaunchKernelGGL(embedding_merge_kernel, dim3((unsigned)(m.groups + f.blocks)), dim3(256), 0, stream, m, f);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  const int64_t piece = piece_of(a.rows, a.cols);
  SumArgs u{a.dY, a.rows, a.cols, a.lddy, a.vocab, keys[from], order[from], (double)a.alpha, a.dW, a.lddw, a.add != nullptr,
            piece, up64(a.rows, piece), reinterpret_cast<double*>(at + lay.parts), part_ld(a.cols), listed + kLists * kListStep, listed, lay.list_ld, (int)up64(a.cols, 64 * kLane), 0};
  e = in_slabs(up64(u.pieces * u.chunks, 4), [&](unsigned grid, int64_t first) {
    u.first = first * 4;
    const dim3 g(grid), b(256);
    if (dtype == DT_F32 && u.onto) hipLaunchKernelGGL((embedding_sum_kernel<float, true>), g, b, 0, stream, u);
    else if (dtype == DT_BF16 && u.onto) hipLaunchKernelGGL((embedding_sum_kernel<bf16_t, true>), g, b, 0, stream, u);
    else if (u.onto) hipLaunchKernelGGL((embedding_sum_kernel<f16_t, true>), g, b, 0, stream, u);
    else if (dtype == DT_F32) hipLaunchKernelGGL((embedding_sum_kernel<float, false>), g, b, 0, stream, u);
    else if (dtype == DT_BF16) hipLaunchKernelGGL((embedding_sum_kernel<bf16_t, false>), g, b, 0, stream, u);
    else hipLaunchKernelGGL((embedding_sum_kernel<f16_t, false>), g, b, 0, stream, u);
  });
  if (e != hipSuccess || u.pieces == 1) return e;
  const int64_t items = up64(u.pieces - 1, kLists) * kLists * u.chunks;
  hipLaunchKernelGGL(embedding_join_kernel, dim3((unsigned)(items < kJoinGroups ? items : kJoinGroups)), dim3(256), 0, stream, u);
  return hipGetLastError();
}

}  // namespace i8g
