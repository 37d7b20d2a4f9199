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
// binary64.  f32 logits are bound by reading them: 8192 x 50304 (1.65 GB, more
// than the 256 MB cache) takes 300 us, 5.5 TB/s, and 20 us more for 4
// alternatives.  2-byte ones are bound by the 14 operations a value, 185 us of
// bf16 being 4.5 TB/s.  The gradient is bound by both reading and writing:
// 4096 x 50257 bf16 (823 MB) 175 us, 4.7 TB/s, where a large copy moves 4.9.
#include "../../include/int8_gemm.h"
#include "i8g_launch.h"
#include "i8g_row.h"

namespace i8g {
namespace {

constexpr int kThreads = 512;                 // of a workgroup of the forward pass
constexpr int kBatch = kThreads * 16;         // columns of a batch: 16 values a thread
constexpr int kPartBatches = 8;               // batches of a part at most: 128 values a thread
constexpr int kMaxParts = 64;                 // parts of a row at most (a wave joins them)
constexpr int kTops = kThreads / 8;           // maxima that a batch leaves, of 8 threads each (kGroup values)
constexpr int kGroup = 128;
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
// The largest of 8 lanes' values, NaN aside.
__device__ __forceinline__ float lanes8_max(float x) {
  x = fmaxf(x, __uint_as_float(lane_partner<1>(__float_as_uint(x))));
  x = fmaxf(x, __uint_as_float(lane_partner<2>(__float_as_uint(x))));
  return fmaxf(x, __uint_as_float(lane_partner<4>(__float_as_uint(x))));
}
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

// Adds a value d = x - m <= 0 to the sums.  2-byte logits are bound by these
// operations, so exp(d) is made of fewer than exp_f32's: ln2 in one part (off
// by 1.9e-9 k), 1 + r q(r) with q of degree 4 (relative error 9.6e-8 for |r| <=
// ln2/2), and an exponent set by one addition, for which d is kept above -87:
// that adds less than 2^-96 to either sum of the longest row.  Off by less
// than (2.6 + 0.05 |d|) 2^-24 relative, and exact for d = 0.  8192 x 50304
// bf16 takes 185 us, with exp_f32 202.
__device__ __forceinline__ void add_value(float& s, float& t, float d) {
  d = __builtin_elementwise_maximum(d, -87.0f);           // (a NaN stays)
  const float big = __builtin_fmaf(d, 1.44269504f, 12582912.0f);
  const float k = big - 12582912.0f;
  const float r = __builtin_fmaf(k, -0.693147182f, d);
  float p = 0x1.0fa83p-7f;
  p = __builtin_fmaf(p, r, 0x1.573a58p-5f);
  p = __builtin_fmaf(p, r, 0x1.555a6ap-3f);
  p = __builtin_fmaf(p, r, 0x1.fffdc6p-2f);
  p = __builtin_fmaf(p, r, 0x1.fffff6p-1f);
  p = __builtin_fmaf(p, r, 1.0f);
  p = __uint_as_float(__float_as_uint(p) + (__float_as_uint(big) << 23));   // (no NaN where d has a payload)
  s += p;
  t = __builtin_fmaf(p, d, t);
}

// With a NaN among its values t is one, and so is s behind this.
__device__ __forceinline__ void keep_nan(float& s, float t) { s += t - t; }

// The outputs of one row from its joined sums (one thread).
struct RowOut {
  double m, log_s;
  bool empty;                                 // no value above -inf: the largest one would add 1
  __device__ __forceinline__ RowOut(const PartSum& p) : m(p.m), log_s(log(p.s)), empty(p.s < 0.5) {}
  __device__ __forceinline__ float log_prob(float x) const {
    return empty ? -__builtin_inff() : (float)((double)x - m - log_s);
  }
};

template <class T>
__device__ __forceinline__ void write_row(const LpArgs& a, int64_t r, const PartSum& p, const RowOut& o) {
  if (a.lse) a.lse[r] = o.empty ? -__builtin_inff() : (float)(o.m + o.log_s);
  if (a.entropy) {
    const double h = o.log_s - p.t / p.s;
    a.entropy[r] = o.empty || h < 0x1p-90 ? 0.0f : (float)h;   // (what add_value adds below -87 is no entropy)
  }
  if (a.logprob) {
    const int64_t t = a.targets[r];
    const bool given = t >= 0 && t < a.cols;
    a.logprob[r] = given ? o.log_prob(to_f32(static_cast<const T*>(a.X)[r * a.ldx + t])) : 0.0f;
  }
}

// The sum over a workgroup of the waves' (s, t) against their maxima.
template <int WAVES>
struct SumLds {
  double s[WAVES], t[WAVES];
  float m[WAVES];
};

// A pass over the logits: the sums of each part of a row, and with TOP the
// maxima of every 8 threads' values of a batch, from which lp_find_kernel or
// lp_join_kernel find the best.  (The values of 8 threads are whole cache
// lines; with a maximum for each thread over all its batches, which are as
// many, reading the best threads' values again took 33 us of 8192 x 50304 f32
// with 4 alternatives, and finding them inside this kernel, whose registers
// and LDS then leave a third of the waves, 50 us, in bf16 117 us.)
template <class T, bool TOP>
__global__ void __launch_bounds__(kThreads) lp_part_kernel(LpArgs a) {
  constexpr int N = kVec<T>, U = 16 / N;      // vectors of a batch: 16 values
  constexpr int WAVES = kThreads / 64;
  __shared__ SumLds<WAVES> red;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = blockIdx.x, lo = part * a.seg;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const int64_t task = r * a.parts + part;
    const int hi = lo + a.seg < a.cols ? lo + a.seg : (int)a.cols;
    const T* row = static_cast<const T*>(a.X) + r * a.ldx;
    float m = kLowest, s = 0.0f, t = 0.0f;
    for (int base = lo; base < hi; base += kThreads * N * U) {
      float v[U][N];
#pragma unroll
      for (int u = 0; u < U; ++u) load_row<T>(row, base + (u * kThreads + tid) * N, hi, -__builtin_inff(), v[u]);
      float b = -__builtin_inff();
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) b = fmaxf(b, v[u][e]);
      if constexpr (TOP) {
        const float top = lanes8_max(b);
        if ((tid & 7) == 0) a.tops[(r * a.batches + base / kBatch) * kTops + (tid >> 3)] = top;
      }
      if (b > m) {
        rescale(s, t, m, b);
        m = b;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) add_value(s, t, v[u][e] - m);
    }
    keep_nan(s, t);
    // join the threads
    float mm = wave_max(m);
    if (lane == 0) red.m[wave] = mm;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) mm = fmaxf(mm, red.m[w]);
    rescale(s, t, m, mm);
    const double ws = wave_sum_f64((double)s), wt = wave_sum_f64((double)t);
    if (lane == 0) {
      red.s[wave] = ws;
      red.t[wave] = wt;
    }
    __syncthreads();
    if (tid == 0) {
      PartSum p{0.0, 0.0, mm};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        p.s += red.s[w];
        p.t += red.t[w];
      }
      if (a.parts > 1) {
        a.sums[task] = LpPart{p.s, p.t, p.m, 0};
      } else {
        const RowOut o(p);
        write_row<T>(a, r, p, o);
        if constexpr (TOP) a.sums[task] = LpPart{o.m, o.log_s, 0.0f, o.empty};
      }
    }
    __syncthreads();                          // LDS is used again
  }
}

// The k best of n candidates in LDS, best first: a candidate's place is the
// number of better ones.  Four lanes count for each, 8 at a time so that the
// reads overlap, until they know that it is not among the best.  `list` has
// room for kPad more, which hold 0.
constexpr int kPad = 31;
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

// What one wave wrote to LDS may be read by its other lanes behind this.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The number of the lane among the set bits of a ballot.
__device__ __forceinline__ int lane_rank(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// The largest bar that at least k keys reach, or one that exactly k reach,
// where at least k reach 1: steps down from the largest key, 4 times as far
// each, then halving.
struct Bar {
  uint32_t bar;
  int n;                                      // keys that reach it
};
template <class F>
__device__ __forceinline__ Bar find_bar(uint32_t top, int k, F reach) {
  uint32_t bar = 0, over = top + 1;           // reached by at least k, by fewer
  int n = 0;
  for (int shift = 20; shift < 32; shift += 2) {
    const uint32_t b = top > 1u << shift ? top - (1u << shift) : 1;
    n = reach(b);
    if (n >= k) {
      bar = b;
      break;
    }
    over = b;
  }
  while (n != k && over - bar > 1) {
    const uint32_t b = bar + (over - bar) / 2;
    const int nb = reach(b);
    if (nb >= k) {
      bar = b;
      n = nb;
    } else {
      over = b;
    }
  }
  return Bar{bar, n};
}

// LDS of one wave's search.
constexpr int kAbove = 256;                   // values above the bar
constexpr int kEqual = 64;                    // and values that equal it, before they are scanned for
constexpr int kSame = 32;                     // groups whose maximum equals the bar, likewise
struct FindLds {
  unsigned long long list[kAbove + kEqual + kPad];
  unsigned short again[kTopMax + kSame];      // groups to read again
  int n_above, n_equal;                       // values noted, above the bar and equal to it
};
constexpr int kChunk = 8 * kBatch;            // columns that one wave searches: 512 groups, 8 a lane

// The end of a chunk that starts at column lo.
__device__ __forceinline__ int chunk_end(const LpArgs& a, int lo) {
  return lo + kChunk < a.cols ? lo + kChunk : (int)a.cols;
}

// What the maxima of a chunk's groups say of its best values.
struct Groups {
  uint32_t bar;                               // a key that at least topk values reach
  int n_again;                                // groups to read again, noted in FindLds::again
  bool few;                                   // whether the groups whose maximum is the bar are among them
};

// By one wave.  The k-th largest of the maxima is a bar that at least k
// values reach, and values above it are only in the at most k groups whose
// maximum is above it.
__device__ __forceinline__ Groups pick_groups(const LpArgs& a, const float* tops, int lo, FindLds& l) {
  constexpr int K = 8;
  const int lane = threadIdx.x & 63, k = a.topk;
  const int n_tops = (chunk_end(a, lo) - lo + kBatch - 1) / kBatch * kTops;   // 64 to 512: at least k
  uint32_t key[K], top = 0;
#pragma unroll
  for (int j = 0; j < K; ++j) key[j] = 64 * j < n_tops ? rank_key(tops[lane + 64 * j]) : 0;
#pragma unroll
  for (int j = 0; j < K; ++j) top = max(top, key[j]);
  top = lanes_max_u32<64>(top);
  auto reach = [&](uint32_t b) __attribute__((always_inline)) {
    int c = 0;
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (64 * j < n_tops) c += __popcll(__ballot(key[j] >= b));
    return c;
  };
  // (a group without values has the key of -inf, so 1 is reached by all)
  const uint32_t bar = find_bar(top, k, reach).bar;
  // the groups above the bar (at most k), then those at it
  int n_again = 0, n_same = 0;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const uint64_t mask = __ballot(key[j] > bar);
    if (key[j] > bar) l.again[n_again + lane_rank(mask)] = (unsigned short)(lane + 64 * j);
    n_again += __popcll(mask);
    n_same += __popcll(__ballot(key[j] == bar));
  }
  const bool few = n_same <= kSame;
  if (few) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const uint64_t mask = __ballot(key[j] == bar);
      if (key[j] == bar) l.again[n_again + lane_rank(mask)] = (unsigned short)(lane + 64 * j);
      n_again += __popcll(mask);
    }
  }
  return Groups{bar, n_again, few};
}

// The values of the groups to read again, by `threads` threads: those above b
// and those equal to it counted in l.n_above and l.n_equal (0 before), and
// with `keep` noted as well, as many as fit, in any order.
template <class T>
__device__ __forceinline__ void scan_groups(const LpArgs& a, const T* row, int lo, FindLds& l, int n_again, uint32_t b,
                                            bool keep, int thread, int threads) {
  constexpr int N = kVec<T>, U = 16 / N;      // vectors of a thread in flight
  constexpr int VECS = kGroup / N;            // of a group, 8 side by side
  const int hi = chunk_end(a, lo), vecs = n_again * VECS;
  const float low = rank_value(b);
  for (int base = 0; base < vecs; base += threads * U) {
    float v[U][N];
    int c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * threads + thread;
      c[u] = hi;                              // (nothing is read there)
      if (i < vecs) {
        const int g = l.again[i / VECS], s = i % VECS;
        c[u] = lo + g / kTops * kBatch + ((s >> 3) * kThreads + g % kTops * 8 + (s & 7)) * N;
      }
      load_row<T>(row, c[u], hi, -__builtin_inff(), v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (v[u][e] < low || c[u] + e >= hi) continue;            // (a NaN may count as -inf)
        const uint32_t x = rank_key(v[u][e]);
        if (x > b) {
          const int i = atomicAdd(&l.n_above, 1);
          if (keep && i < kAbove) l.list[i] = candidate(x, c[u] + e);
        } else if (x == b) {
          const int i = atomicAdd(&l.n_equal, 1);
          if (keep && i < kEqual) l.list[kAbove + i] = candidate(x, c[u] + e);
        }
      }
  }
}

// The min(k, columns) best of the chunk from column lo by one wave, into
// best[0 .. k) (unused places 0): the groups above the bar and at it are read
// again.  If more values are above the bar than fit (many in few groups), the
// bar is raised; if so many equal it that they do not fit (masked rows), the
// ones of lowest index are found by a scan from `lo`.
template <class T>
__device__ __forceinline__ void wave_best(const LpArgs& a, const T* row, const float* tops, int lo, FindLds& l,
                                          unsigned long long* best) {
  constexpr int N = kVec<T>;
  const int lane = threadIdx.x & 63, k = a.topk, hi = chunk_end(a, lo);
  unsigned long long* const equal = l.list + kAbove;
  if (lane < k) best[lane] = 0;
  Groups g = pick_groups(a, tops, lo, l);
  int n_above = 0, n_equal = 0;
  auto scan = [&](uint32_t b, bool keep) __attribute__((always_inline)) {
    if (lane == 0) l.n_above = l.n_equal = 0;
    wave_sync();
    scan_groups<T>(a, row, lo, l, g.n_again, b, keep, lane, 64);
    wave_sync();
    n_above = __builtin_amdgcn_readfirstlane(l.n_above);
    n_equal = __builtin_amdgcn_readfirstlane(l.n_equal);
    wave_sync();
  };
  scan(g.bar, true);
  if (n_above > kAbove) {                     // halving up to a bar with at least k values at or above it
    uint32_t over = 0xFFFFFFFFu;
    while (n_above > kAbove && over - g.bar > 1) {
      const uint32_t b = g.bar + (over - g.bar) / 2;
      const int was = n_above;
      scan(b, false);
      if (n_above + n_equal >= k) {
        g.bar = b;
      } else {
        over = b;
        n_above = was;                        // (of the bar that stays)
      }
    }
    scan(g.bar, true);
  }
  int n = n_above, n_eq = n < k ? n_equal : 0;
  if (n < k && (!g.few || n_eq > kEqual)) {
    const int need = k - n;
    n_eq = 0;
    for (int base = lo; base < hi && n_eq < need; base += 64 * N) {
      const int c = base + lane * N;
      float v[N];
      load_row<T>(row, c, hi, 0.0f, v);
      unsigned int hit = 0;
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (c + e < hi && rank_key(v[e]) == g.bar) hit |= 1u << e;
      int before = __popc(hit);               // inclusive sum over the lanes
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(before, off, 64);
        if (lane >= off) before += o;
      }
      const int total = __shfl(before, 63, 64);
      before += n_eq - __popc(hit);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (hit >> e & 1u) {
          if (before < need) equal[before] = candidate(g.bar, c + e);
          ++before;
        }
      n_eq += total;
    }
    n_eq = n_eq < need ? n_eq : need;
    wave_sync();
  }
  // one list: the equal ones behind the ones above, and padding
  static_assert(kEqual == 64, "one of them a lane");
  const unsigned long long moved = lane < n_eq ? equal[lane] : 0;
  wave_sync();
  if (lane < n_eq) l.list[n + lane] = moved;
  n += n_eq;
  if (lane < kPad) l.list[n + lane] = 0;
  wave_sync();
  place_best(l.list, n, k, best, lane, 64);
  wave_sync();
}

// The best of a row in their order, by `tid` < topk.
__device__ __forceinline__ void write_best(const LpArgs& a, int64_t r, int tid, unsigned long long c, double m,
                                           double log_s, bool empty) {
  const float v = rank_value((uint32_t)(c >> 32));
  a.top_index[r * a.topk + tid] = (int32_t)(0xFFFFFFFFu - (uint32_t)c);
  a.top_logprob[r * a.topk + tid] = empty ? -__builtin_inff() : (float)((double)v - m - log_s);
}

// Rows of one part: a wave a row.  Bound to 8 waves a SIMD, for which f32 keeps
// 2 registers in memory: 8192 x 5000 f32 with 20 alternatives takes 67.6 us
// with the pass over the logits, 73.3 with 7 waves; 8192 x 50304 with 4 312.8
// and 315.0, 1024 x 8192 with 32 25.8 and 25.0.
template <class T>
__global__ void __launch_bounds__(64, 8) lp_find_kernel(LpArgs a) {
  __shared__ FindLds lds;
  __shared__ unsigned long long best[kTopMax];
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const LpPart q = a.sums[r];                 // the row's maximum and log S
    wave_best<T>(a, static_cast<const T*>(a.X) + r * a.ldx, a.tops + r * a.batches * kTops, 0, lds, best);
    if ((int)threadIdx.x < a.topk) write_best(a, r, threadIdx.x, best[threadIdx.x], q.s, q.t, q.empty != 0);
    wave_sync();
  }
}

// Rows of several parts.  Wave 0 joins the sums; of a row of one chunk wave 1
// picks the groups meanwhile, and all waves read them again and rank the
// values (1 x 50257 with 20 alternatives: 11.6 us by one wave alone); of
// longer rows each of the other waves finds the best of a chunk, and all of
// them the best of those.
constexpr int kFinders = 15;
constexpr int kMaxChunks = I8G_VOCAB_MAX / kChunk;
template <class T>
__global__ void __launch_bounds__(64 * (kFinders + 1)) lp_join_kernel(LpArgs a) {
  constexpr int ALL = 64 * (kFinders + 1);
  __shared__ FindLds lds[kFinders];
  __shared__ unsigned long long list[kMaxChunks * kTopMax + kPad];
  __shared__ unsigned long long best[kTopMax];
  __shared__ double row_m, row_l;
  __shared__ int row_empty;
  __shared__ Groups groups;
  static_assert(sizeof(lds) + sizeof(list) + sizeof(best) + 64 <= 65536, "a workgroup's LDS");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int chunks = (a.batches + 7) / 8, n = chunks * a.topk;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const T* row = static_cast<const T*>(a.X) + r * a.ldx;
    const float* tops = a.tops + r * a.batches * kTops;
    if (wave == 0) {
      LpPart q{0.0, 0.0, kLowest, 0};
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
      if (lane < kPad) list[n + lane] = 0;
    } else if (a.topk > 0 && chunks > 1) {
      for (int c = wave - 1; c < chunks; c += kFinders)
        wave_best<T>(a, row, tops + c * 8 * kTops, c * kChunk, lds[wave - 1], list + c * a.topk);
    } else if (a.topk > 0 && wave == 1) {
      const Groups g = pick_groups(a, tops, 0, lds[0]);
      if (lane == 0) {
        groups = g;
        lds[0].n_above = lds[0].n_equal = 0;
      }
    }
    __syncthreads();
    if (a.topk > 0 && chunks > 1) {
      place_best(list, n, a.topk, best, tid, ALL);
    } else if (a.topk > 0) {
      FindLds& l = lds[0];
      scan_groups<T>(a, row, 0, l, groups.n_again, groups.bar, true, tid, ALL);
      __syncthreads();
      const int above = l.n_above, equal = above < a.topk ? l.n_equal : 0;
      if (above <= kAbove && (above >= a.topk || (groups.few && equal <= kEqual))) {
        // both kinds into one list, and padding
        for (int i = tid; i < above + equal + kPad; i += ALL)
          list[i] = i < above ? l.list[i] : i < above + equal ? l.list[kAbove + i - above] : 0;
        __syncthreads();
        place_best(list, above + equal, a.topk, best, tid, ALL);
      } else if (wave == 1) {
        wave_best<T>(a, row, tops, 0, lds[1], best);
      }
    }
    __syncthreads();
    if (tid < a.topk) write_best(a, r, tid, best[tid], row_m, row_l, row_empty);
    __syncthreads();                          // LDS is used again
  }
}

// Short rows: a wave holds a whole row, C values a lane, and finds the best in
// its registers.
constexpr int kShort = 64 * 32;               // columns that one wave takes
constexpr int kShortRows = 4;                 // of a workgroup

// Bound to 4 waves a SIMD up to 32 values a lane, for which 32 in f32 with
// alternatives keep 26 registers in memory: 32768 x 1200 f32 with 5 takes 122
// us, and 173 with the 181 registers and 2 waves that it takes by itself; 8192
// x 2048 with 20 44 and 53, but 1024 x 1500 15.8 and 14.2.
template <class T, int C, bool TOP>
__global__ void __launch_bounds__(64 * kShortRows, C <= 32 ? 4 : 1) lp_short_kernel(LpArgs a) {
  constexpr int N = kVec<T>, U = C / N;
  __shared__ unsigned long long lists[TOP ? kShortRows : 1][kTopMax + kPad];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = (int)a.cols, k = a.topk;
  for (int64_t r = (int64_t)blockIdx.x * kShortRows + wave; r < a.rows; r += (int64_t)gridDim.x * kShortRows) {
    const T* row = static_cast<const T*>(a.X) + r * a.ldx;
    float v[U][N], m = kLowest, s = 0.0f, t = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) load_row<T>(row, (u * 64 + lane) * N, cols, -__builtin_inff(), v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < N; ++e) m = fmaxf(m, v[u][e]);
    m = wave_max(m);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < N; ++e) add_value(s, t, v[u][e] - m);
    keep_nan(s, t);
    const PartSum p{wave_sum_f64((double)s), wave_sum_f64((double)t), m};
    const RowOut o(p);
    if (lane == 0) write_row<T>(a, r, p, o);
    if constexpr (TOP) {
      // The largest bar that k values reach, or one that exactly k reach.
      uint32_t key[U][N], top = 0;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          key[u][e] = (u * 64 + lane) * N + e < cols ? rank_key(v[u][e]) : 0;
          top = max(top, key[u][e]);
        }
      top = lanes_max_u32<64>(top);
      auto reach = [&](uint32_t b) __attribute__((always_inline)) {
        int c = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < N; ++e) c += __popcll(__ballot(key[u][e] >= b));
        return c;
      };
      const Bar bar = find_bar(top, k, reach);
      // Those that reach it if they are k; else those above it, and of those
      // that equal it the ones of lowest index.
      const uint32_t least = bar.n == k ? bar.bar : bar.bar + 1;
      unsigned long long* const list = lists[wave];
      int n = 0;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const uint64_t mask = __ballot(key[u][e] >= least);
          if (key[u][e] >= least) list[n + lane_rank(mask)] = candidate(key[u][e], (u * 64 + lane) * N + e);
          n += __popcll(mask);
        }
      for (int u = 0; u < U && n < k; ++u) {
        int before = n, own = 0;
        uint32_t hit = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          uint32_t x = 0;                     // (registers are not indexed by u)
#pragma unroll
          for (int i = 0; i < U; ++i) x = i == u ? key[i][e] : x;
          const uint64_t mask = __ballot(x == bar.bar);
          before += lane_rank(mask);
          n += __popcll(mask);
          hit |= (x == bar.bar ? 1u : 0u) << e;
        }
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (hit >> e & 1u) {
            if (before + own < k) list[before + own] = candidate(bar.bar, (u * 64 + lane) * N + e);
            ++own;
          }
      }
      if (lane < kPad) list[k + lane] = 0;
      wave_sync();
      // each of the k counts the better ones
      const unsigned long long mine = lane < k ? list[lane] : 0;
      int above = 0;
      for (int j = 0; j < k; j += 8)
#pragma unroll
        for (int e = 0; e < 8; ++e) above += list[j + e] > mine ? 1 : 0;
      if (lane < k) write_best(a, r, above, mine, o.m, o.log_s, o.empty);
      wave_sync();                            // the list is used again
    }
  }
}

// The gradient: a row by `per_row` threads (whole waves, 256 at most) of a
// workgroup of 256, U vectors a thread.
template <class T, int U, bool STREAM>
__global__ void __launch_bounds__(256) lp_bwd_kernel(LpBwdArgs a, int per_row) {
  constexpr int N = kVec<T>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = per_row >> 6;
  const int slot = wave / waves, slots = 4 / waves;
  const int cols = (int)a.cols;
  const int c0 = ((int)blockIdx.x * per_row * U + (int)threadIdx.x - slot * per_row) * N;
  for (int64_t r = (int64_t)blockIdx.y * slots + slot; r < a.rows; r += (int64_t)gridDim.y * slots) {
    const T* x = static_cast<const T*>(a.X) + r * a.ldx;
    T* dx = static_cast<T*>(a.dX) + r * a.lddx;
    float v[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) load_row<T>(x, c0 + u * per_row * N, cols, 0.0f, v[u]);
    // dx_j = -p_j (g + gh (log p_j + H)) = p_j (nh log p_j + n0), and + g for the token
    float lse = a.lse[r], g = 0.0f, n0 = 0.0f, nh = 0.0f;
    int t = -1;
    if (fabsf(lse) >= 16777216.0f) {          // -inf, or so far out that lse is off by 1 and more: p = 0
      lse = __builtin_inff();
    } else {
      if (a.g_logprob) {
        const int64_t token = a.targets[r];
        if (token >= 0 && token < a.cols) {
          t = (int)token;
          g = a.g_logprob[r];
        }
      }
      if (a.g_entropy) nh = -a.g_entropy[r];
      n0 = a.g_entropy ? __builtin_fmaf(nh, a.entropy[r], -g) : -g;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * per_row * N;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float lp = __builtin_elementwise_maximum(v[u][e] - lse, -104.0f);   // p is 0 there, and p * lp as well
        v[u][e] = exp_f32(lp) * __builtin_fmaf(nh, lp, n0);
      }
      if (t >= c && t < c + N) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[u][e] += t == c + e ? g : 0.0f;
      }
      if constexpr (STREAM)
        stream_row<T>(dx, c, cols, v[u]);
      else
        store_row<T>(dx, c, cols, v[u]);
    }
  }
}

// Rows are the grid's y; the workgroups walk on where there are more.
unsigned int row_grid(int64_t rows) { return (unsigned int)(rows < 65535 ? rows : 65535); }

template <class T, int C, bool TOP>
hipError_t forward_short(const LpArgs& a, hipStream_t stream) {
  const int64_t most = int64_t(1) << 20, groups = (a.rows + kShortRows - 1) / kShortRows;
  const dim3 grid((unsigned int)(groups < most ? groups : most)), block(64 * kShortRows);
  if constexpr (TOP)
    if (a.topk > 0) {
      hipLaunchKernelGGL((lp_short_kernel<T, C, true>), grid, block, 0, stream, a);
      return hipGetLastError();
    }
  hipLaunchKernelGGL((lp_short_kernel<T, C, false>), grid, block, 0, stream, a);
  return hipGetLastError();
}

// Rows of up to 2048 columns by a wave each (by the kernels of longer rows in
// parentheses, bf16): 32768 x 1000 29.6 us (148), with 5 alternatives 63 (160);
// 128 x 1500 with 20 alternatives 20.0 (18.2), with 32 21.0 (39.2), where a
// batch leaves fewer maxima than that; 1 x 1000 3.3 (3.8).  Up to 4096 where
// nothing is searched for and there are rows for every SIMD: 8192 x 4096 22.5
// (37.4), 1024 x 4096 6.3 (7.2), 128 x 4096 6.3 (4.3); 8192 x 8192 53 (48).
template <class T>
hipError_t forward(const LpArgs& a, hipStream_t stream) {
  if (a.cols <= 64 * 8) return forward_short<T, 8, true>(a, stream);
  if (a.cols <= 64 * 16) return forward_short<T, 16, true>(a, stream);
  if (a.cols <= kShort) return forward_short<T, 32, true>(a, stream);
  if (a.cols <= 2 * kShort && a.topk == 0 && a.rows >= 1024) return forward_short<T, 64, false>(a, stream);
  const dim3 grid(a.parts, row_grid(a.rows)), block(kThreads);
  if (a.topk > 0)
    hipLaunchKernelGGL((lp_part_kernel<T, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((lp_part_kernel<T, false>), grid, block, 0, stream, a);
  if (a.parts > 1) {
    hipLaunchKernelGGL((lp_join_kernel<T>), dim3(1, row_grid(a.rows)), dim3(64 * (kFinders + 1)), 0, stream, a);
  } else if (a.topk > 0) {
    const int64_t most = int64_t(1) << 20;
    hipLaunchKernelGGL((lp_find_kernel<T>), dim3((unsigned int)(a.rows < most ? a.rows : most)), dim3(64), 0, stream, a);
  }
  return hipGetLastError();
}

template <class T, int U>
hipError_t backward(const LpBwdArgs& a, int per_row, hipStream_t stream) {
  const int chunk = per_row * kVec<T> * U, slots = 256 / per_row;
  const dim3 grid((unsigned int)((a.cols + chunk - 1) / chunk), row_grid((a.rows + slots - 1) / slots));
  // a gradient larger than half the last-level cache is stored around it
  if ((double)a.rows * (double)a.cols * sizeof(T) > kStreamOutBytes)
    hipLaunchKernelGGL((lp_bwd_kernel<T, U, true>), grid, dim3(256), 0, stream, a, per_row);
  else
    hipLaunchKernelGGL((lp_bwd_kernel<T, U, false>), grid, dim3(256), 0, stream, a, per_row);
  return hipGetLastError();
}

// Two vectors a thread (4096 x 50304 f32 272 us; 301 with four, 327 with one);
// one where 256 threads then hold the row, and one or two waves where they do
// (32768 x 1000 bf16 by 128 threads 28.6 us; by 256 41 us, with two vectors 60).
template <class T>
hipError_t backward(const LpBwdArgs& a, hipStream_t stream) {
  const int64_t vecs = (a.cols + kVec<T> - 1) / kVec<T>;
  if (vecs > 256) return backward<T, 2>(a, 256, stream);
  return backward<T, 1>(a, vecs <= 64 ? 64 : vecs <= 128 ? 128 : 256, stream);
}

}  // namespace

// Parts of a row, of whole batches: as many as its length needs, and with few
// rows as many as fill the chip.  (None of a row that a wave holds.)
LpSplit lp_split(int64_t rows, int64_t cols) {
  if (cols <= kShort) return LpSplit{0, 0, 0, 0};
  const int64_t batches = (cols + kBatch - 1) / kBatch;
  const int64_t need = (batches + kPartBatches - 1) / kPartBatches;
  const int64_t fill = rows >= 512 ? 1 : (512 + rows - 1) / rows;
  int64_t parts = fill < need ? need : fill < batches ? fill : batches;
  if (parts > kMaxParts) parts = kMaxParts;
  const int64_t each = (batches + parts - 1) / parts;
  return LpSplit{(int)((batches + each - 1) / each), (int)(each * kBatch), (int)batches, (size_t)batches * kTops};
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
