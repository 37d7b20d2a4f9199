// head.hip -- log probabilities of given tokens straight from the int8
// operands of the LM head's product, and the gradients of both operands.  The
// logits are never stored.
//
// With L_ij = RN(RN(RN(acc_ij) s_row_i) s_col_j), acc = QA . QBt^T (the value
// that gemm_i8_blockscaled writes):
//   lse_i = log sum_j exp L_ij            logprob_i = L_it - lse_i
//   G_ij = g_i ([j = t] - p_ij) + gl_i p_ij,   p_ij = exp(L_ij - lse_i)
//   dA_ik = sum_j G_ij s_col_j QBt_jk     dBt_jk = sum_i G_ij s_row_i QA_ik
// Both gradients read one matrix T_ij = s_row_i G_ij s_col_j:
//   dA_ik = (1 / s_row_i) sum_j T_ij QBt_jk,  dBt_jk = (1 / s_col_j) sum_i T_ij QA_ik,
// and the codes are exact in bf16.  T goes to the matrix cores as a sum of bf16
// terms: three for f32 and f16 gradients, which hold all 24 bits of a binary32
// number, and two for bf16 ones (2^-16 of each value, where the outputs' own
// rounding is 2^-8).  bf16 has binary32's exponents, so a probability of 2^-120 has
// as many bits as one of 1/2: a rare token's row of dBt is nothing but such values.
// (f16 terms are half the products, or two thirds, but their least number is a
// probability of 2^-40.)  Powers of two of each row and column keep the scales from mattering (see
// the backward part).
//
// Forward: a workgroup multiplies a tile of vocabulary rows by a tile of
// tokens; the vocabulary is the accumulators' row dimension, so that a lane
// holds one token's logits and a row's maximum and sum are in-lane work.  A
// tile leaves (max, sum) of its part of every row; a second kernel joins them
// and computes the given token's logit anew.
// Backward: in pieces of the vocabulary.  A piece's tiles are multiplied again
// and leave T in blocks of 32 tokens by 16 vocabulary rows, 1 KiB each, in the
// register order of the matrix cores' operands: dA's product reads a block as
// it is, dBt's through the transposing LDS read.  Both products of a piece run
// in one launch.
#include "../../include/int8_gemm.h"
#include "i8g_launch.h"
#include "i8g_row.h"

#include <type_traits>
#include <utility>

namespace i8g {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269502f;
constexpr float kLowest = -3.40282347e38f;   // the running maximum's start: finite, so that x - m is no NaN for a finite x or -inf

template <int N>
__device__ __forceinline__ void wait_loads() {   // all but the last N vector loads, and every LDS access
  static_assert(N >= 0 && N < 64, "vmcnt is a 6-bit counter");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (((N >> 4) & 3) << 14));
}
// Workgroup barrier without the memory fence of __syncthreads(), which would
// wait for the loads in flight; callers wait for what they need first.
__device__ __forceinline__ void barrier_nofence() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// Direct loads of 16 bytes a lane to lds + 16 * lane.  The compiler makes LDS
// reads wait for every direct load in flight that it knows of, and would empty
// the pipeline at each stage, so these are not told to it: nothing returns to a
// register, and the callers wait.  (m0, which holds the destination, has no
// other use in these kernels: the compiler writes it for direct loads and
// indexed registers only.)
__device__ __forceinline__ uint32_t lds_address(const int8_t* lds) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const int8_t*)lds;
}
__device__ __forceinline__ void lds_load16(const int8_t* g, const int8_t* lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds_address(lds)), "v"(g)
               : "memory");
}
__device__ __forceinline__ void lds_load16(const char* base, int offset, const int8_t* lds) {   // base: uniform
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds_address(lds)), "v"(offset), "s"(base)
               : "memory");
}
__device__ __forceinline__ void lds_load4(const void* g, const void* lds) {     // 4 bytes a lane to lds + 4 * lane
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds_address(static_cast<const int8_t*>(lds))), "v"(g)
               : "memory");
}
// Asks for the READS fragment reads of the next k-step between this one's
// MFMAs, one by one.
template <int READS, int MFMAS>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int t = 0; t < (READS < MFMAS ? READS : MFMAS); ++t) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
  }
  if constexpr (READS < MFMAS) __builtin_amdgcn_sched_group_barrier(0x008, MFMAS - READS, 0);
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ float other_half(float x) {   // the value of lane ^ 32
  const Pair32 p = lane_pair<32>(__float_as_uint(x));
  return __uint_as_float(threadIdx.x & 32 ? p.a : p.b);
}

// ---- the logits of a tile -----------------------------------------------------
struct LogitArgs {
  const int8_t *A, *B;         // tokens x K, vocab x K
  const float *s_row, *s_col;
  int64_t lda, ldb;
  int M, N, K;
};

// BV vocabulary rows by BT tokens, WV x WT waves; stages of SB bytes of K, S of
// them in LDS, filled by direct loads (16-byte chunk c of row r at c ^ (r/2)%8, or c
// ^ (r/4)%4 of 64 bytes, which spreads a fragment's 32 rows over the banks).
template <int BV, int BT, int WV, int WT, int SB = 128, int S = 2>
struct LogitTile {
  static constexpr int NW = WV * WT, NT = NW * 64;
  static constexpr int FV = BV / WV / 32, FT = BT / WT / 32;
  static constexpr int CH = SB / 16, KS = SB / 32, ROWS = 64 / CH;   // chunks and k-steps of a stage, rows of a load
  static constexpr int STAGE = (BV + BT) * SB;
  static constexpr int INS = (BV + BT) / (ROWS * NW), INS_V = BV / (ROWS * NW);
  static_assert(INS * ROWS * NW == BV + BT && INS_V * ROWS * NW == BV && NW % 2 == 0 && (SB == 128 || SB == 64), "whole loads");
  static constexpr int LDS = S * STAGE;
  static __device__ __forceinline__ int turn_of(int row) { return SB == 128 ? (row >> 1) & 7 : (row >> 2) & 3; }
  static constexpr int TOKENS = BT < 64 ? 64 : BT;         // values of a token in LDS: whole waves' loads

  // Where a lane's loads of a tile begin: rows (q * NW + wave) * ROWS + lane / CH;
  // NW is even, so a row's turn does not depend on q.
  struct Source {
    const int8_t* at[INS];
  };
  static __device__ __forceinline__ int wave_of() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
  static __device__ __forceinline__ void issue(const LogitArgs& p, int8_t* smem, const Source& src, int kt) {
    const int lane = threadIdx.x & 63, wave = wave_of();
    const int chunk = (lane & (CH - 1)) ^ turn_of(wave * ROWS + lane / CH);
    int8_t* base = smem + kt % S * STAGE + wave * 1024;
    const int at = min(kt * SB + chunk * 16, ((p.K + 15) & ~15) - 16);   // (what lies beyond K is cleared below)
#pragma unroll
    for (int q = 0; q < INS; ++q) lds_load16(src.at[q] + at, base + q * NW * 1024);
  }
  // n values of 4 bytes from `first` on into LDS, the last of `all` again behind them.
  template <int n>
  static __device__ __forceinline__ void load_values(const void* from, int64_t first, int64_t all, void* lds) {
    const int lane = threadIdx.x & 63;
    for (int i = wave_of(); i < n / 64; i += NW) {
      const int64_t at = first + i * 64 + lane;
      lds_load4(static_cast<const float*>(from) + (at < all ? at : all - 1), static_cast<float*>(lds) + i * 64);
    }
  }
  // The first S stages of a tile, into LDS that no wave reads any more.
  static __device__ __forceinline__ void start(const LogitArgs& p, int8_t* smem, int v0, int t0, Source& src) {
    const int lane = threadIdx.x & 63, wave = wave_of();
#pragma unroll
    for (int q = 0; q < INS; ++q) {
      const int r = (q * NW + wave) * ROWS + lane / CH;
      if (q < INS_V) src.at[q] = p.B + (int64_t)min(v0 + r, p.N - 1) * p.ldb;
      else src.at[q] = p.A + (int64_t)min(t0 + r - BV, p.M - 1) * p.lda;
    }
#pragma unroll
    for (int st = 0; st < S; ++st)
      if (p.K > st * SB) issue(p, smem, src, st);
  }

  // What this wave asked for up to start() is waited for here, but not the BEHIND vector stores
  // that this wave has issued after it where `behind` says so.
  template <int BEHIND>
  static __device__ __forceinline__ void multiply(const LogitArgs& p, int8_t* smem, const Source& src, bool behind,
                                                  v16i (&acc)[FV][FT]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_of();
    const int wv = wave / WT, wt = wave % WT;
    const int n = (p.K + SB - 1) / SB;
#pragma unroll
    for (int i = 0; i < FV; ++i)
#pragma unroll
      for (int j = 0; j < FT; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
    if (n == 0) {
      wait_loads<0>();
      barrier_nofence();
      return;
    }
    // The last stage's bytes beyond K: cleared in the tokens' rows, which makes
    // those products 0 whatever the other operand's bytes are.
    auto clear_tail = [&](int kt) {
      const int left = p.K - kt * SB;
      if (left >= SB) return;
      int8_t* base = smem + kt % S * STAGE + BV * SB;
      for (int c = tid; c < BT * CH; c += NT) {
        const int r = c / CH, first = c % CH * 16;
        if (first + 16 <= left) continue;
        uint32_t* w = reinterpret_cast<uint32_t*>(base + r * SB + (c % CH ^ turn_of(r)) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int keep = left - first - 4 * i;             // bytes of this word that are kept
          if (keep <= 0) w[i] = 0;
          else if (keep < 4) w[i] &= (1u << (8 * keep)) - 1;
        }
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);                    // lgkmcnt(0)
      barrier_nofence();
    };

    int offv[KS][FV], offt[KS][FT];
    const int half = lane >> 5;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
#pragma unroll
      for (int i = 0; i < FV; ++i) {
        const int r = (wv * FV + i) * 32 + (lane & 31);
        offv[s][i] = r * SB + ((2 * s + half) ^ turn_of(r)) * 16;
      }
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        const int r = BV + (wt * FT + j) * 32 + (lane & 31);
        offt[s][j] = r * SB + ((2 * s + half) ^ turn_of(r)) * 16;
      }
    }
    auto read = [&](int kt, int s, v4i (&fv)[FV], v4i (&ft)[FT]) {
      const int8_t* base = smem + kt % S * STAGE;
#pragma unroll
      for (int i = 0; i < FV; ++i) fv[i] = *reinterpret_cast<const v4i*>(base + offv[s][i]);
#pragma unroll
      for (int j = 0; j < FT; ++j) ft[j] = *reinterpret_cast<const v4i*>(base + offt[s][j]);
    };
    auto mfma = [&](const v4i (&fv)[FV], const v4i (&ft)[FT]) {
#pragma unroll
      for (int i = 0; i < FV; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fv[i], ft[j], acc[i][j], 0, 0, 0);
    };
    v4i fv0[FV], ft0[FT], fv1[FV], ft1[FT];
    if (n < S) wait_loads<0>();
    else if (BEHIND > 0 && behind) wait_loads<INS * (S - 1) + BEHIND>();
    else wait_loads<INS * (S - 1)>();
    barrier_nofence();
    if (n == 1) clear_tail(0);
    read(0, 0, fv0, ft0);
    const auto steps = [&](int kt) {                         // all of a stage but the last
#pragma unroll
      for (int s = 0; s + 2 < KS; s += 2) {
        read(kt, s + 1, fv1, ft1);
        mfma(fv0, ft0);
        interleave<FV + FT, FV * FT>();
        read(kt, s + 2, fv0, ft0);
        mfma(fv1, ft1);
        interleave<FV + FT, FV * FT>();
      }
      read(kt, KS - 1, fv1, ft1);
      mfma(fv0, ft0);
      interleave<FV + FT, FV * FT>();
    };
    // (the last stage stands apart: a branch around the products would move the
    // accumulators)
    for (int kt = 0; kt + 1 < n; ++kt) {
      steps(kt);
      // the next stage has landed, and this one's last fragments are in
      // registers: its buffer is free
      if (S > 2 && kt + S <= n) wait_loads<INS * (S - 2)>();
      else wait_loads<0>();
      barrier_nofence();
      if (kt + S < n) issue(p, smem, src, kt + S);
      if (kt + 2 == n) clear_tail(kt + 1);
      read(kt + 1, 0, fv0, ft0);
      mfma(fv1, ft1);
      interleave<FV + FT, FV * FT>();
    }
    steps(n - 1);
    mfma(fv1, ft1);
  }
};

// ---- forward --------------------------------------------------------------------
struct FwdArgs {
  LogitArgs l;
  int v0;                      // first vocabulary row
  int tiles_v, tiles_t;
  v2f* parts;                  // [tiles_v][M]: the maximum, and the sum of exp(x - maximum)
};

// The tiles of a workgroup: an XCD (workgroups are dealt to the 8 in turn) takes
// an eighth of the tiles, neighbours in their order, its workgroups every so
// many.  Where a workgroup has several, the next one's first loads are on their
// way while this one's logits are worked on (8192 x 50304 x 768: 377 us, and 385
// with a workgroup a tile).
struct Walk {
  int at, end, step;
  __device__ Walk(int first, int total, int tiles) {       // tiles first ... first + total - 1 of `tiles`
    const int xcd = blockIdx.x & 7;
    const int n = min(total, tiles - first);
    at = first + (int)((int64_t)n * xcd / 8) + (int)(blockIdx.x >> 3);
    end = first + (int)((int64_t)n * (xcd + 1) / 8);
    step = (int)(gridDim.x >> 3);
  }
};
// Tiles of tokens that share a vocabulary tile in an L2 before the next one.
constexpr int kGroupT = 8;
__device__ __forceinline__ void tile_of(int w, int tiles_v, int tiles_t, int& tv, int& tt) {
  const int group = w / (kGroupT * tiles_v), first = group * kGroupT;
  const int wide = min(kGroupT, tiles_t - first), in = w - group * kGroupT * tiles_v;
  tt = first + in % wide;
  tv = in / wide;
}

// A tile's (max, sum) of each of its tokens.  8192 x 50304 x 768: 380 us, 1.66
// POPS (a library's 8192^3 int8 product reaches 2.05).  The products and their
// LDS reads alone take 264, the logits' part behind them 100: accumulators and
// fragments fill the registers, so one tile's logits cannot go beside the next
// one's products.  (128 x 128 with two workgroups a CU 406 us, four waves of 128 x
// 128 490.)  One token: 8.5 us for 38.6 MB of codes, 4.5 TB/s.
template <int BV, int BT, int WV, int WT, int PER_CU, int SB = 128, int S = 2>
__global__ void __launch_bounds__(WV * WT * 64, PER_CU * WV * WT / 4) head_fwd_kernel(const FwdArgs p) {
  using Tile = LogitTile<BV, BT, WV, WT, SB, S>;
  constexpr int FV = Tile::FV, FT = Tile::FT;
  __shared__ __attribute__((aligned(1024))) int8_t smem[Tile::LDS];
  __shared__ __attribute__((aligned(16))) float sc[2][BV], rows[2][Tile::TOKENS];
  __shared__ v2f part[WV][BT];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wv = wave / WT, wt = wave % WT;
  Walk walk(0, p.tiles_v * p.tiles_t, p.tiles_v * p.tiles_t);
  if (walk.at >= walk.end) return;
  int tv, tt;
  tile_of(walk.at, p.tiles_v, p.tiles_t, tv, tt);
  typename Tile::Source src;
  const auto start = [&](int turn) {
    Tile::template load_values<BV>(p.l.s_col, p.v0 + tv * BV, p.l.N, sc[turn]);
    Tile::template load_values<Tile::TOKENS>(p.l.s_row, tt * BT, p.l.M, rows[turn]);
    Tile::start(p.l, smem, p.v0 + tv * BV, tt * BT, src);
  };
  start(0);
  for (int turn = 0;; turn ^= 1) {
    const int v0 = p.v0 + tv * BV, t0 = tt * BT, tile_v = tv;
    v16i acc[FV][FT];
    Tile::template multiply<0>(p.l, smem, src, false, acc);
    walk.at += walk.step;
    const bool more = walk.at < walk.end;
    if (more) {
      barrier_nofence();                                   // every wave has read this tile's last fragments
      tile_of(walk.at, p.tiles_v, p.tiles_t, tv, tt);
      start(turn ^ 1);
    }
    const float* scale = sc[turn];
    const int half = lane >> 5;
    const bool ragged = v0 + BV > p.l.N;
#pragma unroll
    for (int j = 0; j < FT; ++j) {
      const float sr = rows[turn][(wt * FT + j) * 32 + (lane & 31)];
      float x[FV][16];
      float m = kLowest;
#pragma unroll
      for (int i = 0; i < FV; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = (wv * FV + i) * 32 + 8 * q + 4 * half;
          const v4f s4 = *reinterpret_cast<const v4f*>(scale + r);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = epilogue1(acc[i][j][4 * q + e], sr, s4[e]);
            if (ragged && v0 + r + e >= p.l.N) y = -__builtin_inff();
            x[i][4 * q + e] = y;
            m = fmaxf(m, y);
          }
        }
      m = fmaxf(m, other_half(m));
      // exp(x - m) as 2^(x c - m2), c = log2 e and m2 = RN(m c): one fused step,
      // and one factor for m2's rounding; where that rounding may be more than a
      // factor of two, the difference by itself (in these lanes only: a row's
      // bits do not depend on another's)
      const float m2 = m * kLog2e;
      const bool far = !(fabsf(m2) < 16777216.0f);
      float s = 0.0f;
      if (__builtin_amdgcn_ballot_w64(far) == 0) {
#pragma unroll
        for (int i = 0; i < FV; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) s += __builtin_amdgcn_exp2f(__builtin_fmaf(x[i][e], kLog2e, -m2));
      } else {
#pragma unroll
        for (int i = 0; i < FV; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            s += __builtin_amdgcn_exp2f(far ? (x[i][e] - m) * kLog2e : __builtin_fmaf(x[i][e], kLog2e, -m2));
      }
      if (!far) s *= __builtin_amdgcn_exp2f(-__builtin_fmaf(m, kLog2e, -m2));
      s += other_half(s);
      if (half == 0) part[wv][(wt * FT + j) * 32 + lane] = v2f{m, s};
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);                      // lgkmcnt(0)
    barrier_nofence();
    if (tid < BT && t0 + tid < p.l.M) {
      v2f a = part[0][tid];
#pragma unroll
      for (int w = 1; w < WV; ++w) {
        const v2f b = part[w][tid];
        const float m = fmaxf(a.x, b.x);
        a.y = a.y * __builtin_amdgcn_exp2f((a.x - m) * kLog2e) + b.y * __builtin_amdgcn_exp2f((b.x - m) * kLog2e);
        a.x = m;
      }
      p.parts[(size_t)tile_v * p.l.M + t0 + tid] = a;
    }
    if (!more) return;
  }
}

struct JoinArgs {
  LogitArgs l;
  const int64_t* targets;
  const v2f* parts;
  int n_parts;
  float *logprob, *lse;        // may be null
};

// R rows a workgroup: 256 / R threads a row join its parts, then a wave a row
// computes the given token's logit.  Latency: the row's maximum,
// then its sums, then the token's codes wait for each other; 393 parts of a row 4
// us, 8192 rows of some 200 10 us (13 MB).
template <int R>
__global__ void __launch_bounds__(256) head_join_kernel(const JoinArgs p) {
  constexpr int S = 256 / R;
  __shared__ double sum[S][R];
  __shared__ float top[S][R];
  __shared__ float out[R];
  const int tid = threadIdx.x, r = tid % R, slot = tid / R;
  const int row = blockIdx.x * R + r;
  // maxima are finite or +inf, never NaN (they ignore it; the sum is NaN then)
  float m = kLowest;
  if (row < p.l.M)
#pragma unroll 4
    for (int i = slot; i < p.n_parts; i += S) m = fmaxf(m, p.parts[(size_t)i * p.l.M + row].x);
  top[slot][r] = m;
  __syncthreads();
#pragma unroll
  for (int d = S / 2; d >= 1; d >>= 1) {
    if (slot < d) top[slot][r] = fmaxf(top[slot][r], top[slot + d][r]);
    __syncthreads();
  }
  m = top[0][r];
  double s = 0.0;
  if (row < p.l.M)
#pragma unroll 4
    for (int i = slot; i < p.n_parts; i += S) {
      const v2f a = p.parts[(size_t)i * p.l.M + row];
      s += (double)(a.y * __builtin_amdgcn_exp2f((a.x - m) * kLog2e));
    }
  sum[slot][r] = s;
  __syncthreads();
#pragma unroll
  for (int d = S / 2; d >= 1; d >>= 1) {
    if (slot < d) sum[slot][r] += sum[slot + d][r];
    __syncthreads();
  }
  if (slot == 0) {
    // the largest logit's share is 1: roundings below it would put a logprob above 0
    // (a sum of 0: every logit is -inf)
    const double all = sum[0][r];
    const float lse = (float)((double)m + log(all > 0.0 && all < 1.0 ? 1.0 : all));
    out[r] = lse;
    if (row < p.l.M && p.lse) p.lse[row] = lse;
  }
  if (!p.logprob) return;
  __syncthreads();
  const int lane = tid & 63;
  for (int i = tid >> 6; i < R; i += 4) {
    const int at = blockIdx.x * R + i;
    if (at >= p.l.M) return;
    const int64_t t = p.targets[at];
    float lp = 0.0f;
    if (t >= 0 && t < p.l.N) {
      const int8_t *a = p.l.A + (int64_t)at * p.l.lda, *b = p.l.B + t * p.l.ldb;
      int acc = 0;
      for (int k = lane * 16; k < p.l.K; k += 1024) {
        v4i x = *reinterpret_cast<const v4i*>(a + k);
        const v4i y = *reinterpret_cast<const v4i*>(b + k);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int keep = p.l.K - k - 4 * w;
          if (keep < 4) x[w] = keep <= 0 ? 0 : x[w] & ((1 << (8 * keep)) - 1);
          acc = __builtin_amdgcn_sdot4(x[w], y[w], acc, false);
        }
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) acc += __shfl_xor(acc, d, 64);
      const float x = epilogue1(acc, p.l.s_row[at], p.l.s_col[t]), lse = out[i];
      lp = lse == -__builtin_inff() ? lse : x - lse;         // (every logit -inf: so is every log probability)
    }
    if (lane == 0) p.logprob[at] = lp;
  }
}

// ---- backward ---------------------------------------------------------------------
// Powers of two.  With r = |g_i| + |gl_i|, a row's (|g| + |gl|) s_row is below
// 2^(exponent r + exponent s_row), E of the rows at most, and s_col below its
// power, F at most.  T_ij is multiplied by 2^(kTop - E + a_i - F + b_j), where a_i
// and b_j are how far the row and the column are below E and F, and the codes of
// row i (j) by 2^-a_i (2^-b_j), which is exact: a_i and b_j are kMostShift at most,
// and bf16 goes down to 2^-126.  So T is of the size of p, whatever the scales and
// gradients are: rows of small numbers (of zeros, whose scale is the least one)
// have gradients as exact as others.  |T| is at most 2^kTop, times what the
// rounding of a log-sum-exp below 2^24 makes of p, 1.65 at most: the least p, 2^-126,
// leaves T's low terms 2^-79, and 2^30 products with codes stay below 2^102.
constexpr int kBounds = 64, kMostShift = 100, kTop = 64;
struct Bound {
  uint32_t row, col;           // E + 1024 and F + 1024 of a part, 0: none
};
struct Scale {                 // acc m 2^x is the gradient: m = RN(1 / mantissa) of the row's scale
  float m;
  int x;
  __device__ float of(float acc) const { return __builtin_ldexpf(acc * m, x); }
};
struct RowArgs {
  const int64_t* targets;
  const float *g, *gl, *s_row, *s_col;
  int M, N;
};
struct TokenRow {
  float g, gl, s;              // g 0 for a row without a token
  int eg, es;
  __device__ TokenRow(const RowArgs& p, int64_t i) : g(0.0f), gl(p.gl ? p.gl[i] : 0.0f), s(p.s_row[i]) {
    if (p.g) {
      const int64_t t = p.targets[i];
      const float at_t = p.g[i];
      g = t >= 0 && t < p.N ? at_t : 0.0f;
    }
    eg = __builtin_amdgcn_frexp_expf(fabsf(g) + fabsf(gl));
    es = __builtin_amdgcn_frexp_expf(s);
  }
  __device__ uint32_t bound() const {            // (of a finite row that has a gradient)
    const float r = fabsf(g) + fabsf(gl);
    return r > 0.0f && r < __builtin_inff() && s > 0.0f && s < __builtin_inff() ? (uint32_t)(eg + es + 1024) : 0u;
  }
};
__device__ __forceinline__ uint32_t col_bound(float s) {
  return s > 0.0f && s < __builtin_inff() ? (uint32_t)(__builtin_amdgcn_frexp_expf(s) + 1024) : 0u;
}
// Of a workgroup's part of the rows; the same in all its threads.
__device__ Bound bound_of(const RowArgs& p, int part, int parts) {
  __shared__ uint32_t most[2][4];
  const int tid = threadIdx.x;
  uint32_t row = 0, col = 0;
  const int64_t first = (int64_t)part * 256 + tid, step = parts * 256;
  for (int64_t i = first; i < p.M; i += 4 * step)          // (the last row's again behind it)
#pragma unroll
    for (int q = 0; q < 4; ++q) row = max(row, TokenRow(p, min(i + q * step, (int64_t)p.M - 1)).bound());
  for (int64_t j = first; j < p.N; j += 4 * step)
#pragma unroll
    for (int q = 0; q < 4; ++q) col = max(col, col_bound(p.s_col[min(j + q * step, (int64_t)p.N - 1)]));
  row = lanes_max_u32<64>(row);
  col = lanes_max_u32<64>(col);
  most[0][tid >> 6] = row;
  most[1][tid >> 6] = col;
  __syncthreads();
  return Bound{max(max(most[0][0], most[0][1]), max(most[0][2], most[0][3])),
               max(max(most[1][0], most[1][1]), max(most[1][2], most[1][3]))};
}
__global__ void __launch_bounds__(256) head_bounds_kernel(const RowArgs p, Bound* bounds) {
  const Bound b = bound_of(p, blockIdx.x, kBounds);
  if (threadIdx.x == 0) bounds[blockIdx.x] = b;
}

// Before the pieces: both operands' codes as bf16 blocks of 16 rows (the
// contraction) by 32 columns, 1 KiB in the order of a fragment: lane l holds
// column l%32, rows 8 (l/32) ... + 7.  Zero beyond the rows and `cols`.  And what
// the products need of each row.
// Up to so many rows of both sides every workgroup looks through them itself, and
// no launch comes before (805 x 1864 x 296 takes 1.3 us less than with it, 1500 x
// 6000 x 100 1.8 more).
constexpr int kOwnBounds = 4096;
struct PackArgs {
  LogitArgs l;
  RowArgs rows;
  const Bound* bounds;         // null: each workgroup's own
  int blocks_a, blocks_b;      // blocks of 16 rows
  int KB;                      // blocks of 32 columns
  v4i* out;                    // [blocks][KB][64]: tokens, vocabulary rows
  float *share, *given;        // of a token, in T: (gl - g) s_row and g s_row times their power of two
  float* col;                  // of a vocabulary row, in T: s_col times its power of two
  Scale *scale_a, *scale_b;
};
// 8192 x 50304 x 768: 45 MB read, 90 MB written in 26 us, and 45 where a thread
// stores its 64 bytes itself: they go through LDS, within the wave, so that a
// store has a block's whole KiB.
__global__ void __launch_bounds__(256) head_prepare_kernel(const PackArgs p) {
  const int tid = threadIdx.x;
  Bound most;
  if (p.bounds) {
    most = p.bounds[tid & 63];
    most.row = lanes_max_u32<64>(most.row);
    most.col = lanes_max_u32<64>(most.col);
  } else {
    most = bound_of(p.rows, 0, 1);
  }
  const int E = most.row ? (int)most.row - 1024 : 0, F = most.col ? (int)most.col - 1024 : 0;
  const int c4 = tid & 7, half = (tid >> 3) & 1;           // 16 threads a block, 4 columns and 8 rows each
  const int64_t blocks = (int64_t)(p.blocks_a + (int64_t)p.blocks_b) * p.KB;
  __shared__ __attribute__((aligned(16))) v4i lds[4][256];
  const int lane = tid & 63, wave = tid >> 6;
  for (int64_t at0 = (int64_t)blockIdx.x * 16 + wave * 4; at0 < blocks; at0 += (int64_t)gridDim.x * 16) {
    const int64_t at = min(at0 + (lane >> 4), blocks - 1);
    const bool a = at < (int64_t)p.blocks_a * p.KB;
    const int64_t block = a ? at : at - (int64_t)p.blocks_a * p.KB;
    const int8_t* Q = a ? p.l.A : p.l.B;
    const int64_t ld = a ? p.l.lda : p.l.ldb;
    const int rows = a ? p.l.M : p.l.N;
    const int64_t b16 = block / p.KB;
    const int kb = (int)(block - b16 * p.KB);
    const int k = kb * 32 + c4 * 4;
    // the 8 threads of a half have a row each
    const int64_t own = b16 * 16 + half * 8 + c4;
    int shift = 0;
    if (a && own < rows) {
      const TokenRow r(p.rows, own);
      const int below = E - r.eg - r.es;
      shift = min(max(below, 0), kMostShift);
      if (kb == 0) {
        const float f = __builtin_ldexpf(r.s, kTop - r.es + min(shift - below, 0));
        p.share[own] = __builtin_ldexpf(r.gl - r.g, -r.eg) * f;
        p.given[own] = __builtin_ldexpf(r.g, -r.eg) * f;
        p.scale_a[own] = Scale{1.0f / __builtin_amdgcn_frexp_mantf(r.s), E + F - kTop - shift - r.es};
      }
    } else if (own < rows) {
      const float c = p.l.s_col[own];
      const int e = __builtin_amdgcn_frexp_expf(c);
      shift = min(max(F - e, 0), kMostShift);
      if (kb == 0) {
        p.col[own] = __builtin_ldexpf(c, shift - F);
        p.scale_b[own] = Scale{1.0f / __builtin_amdgcn_frexp_mantf(c), E + F - kTop - shift - e};
      }
    }
    const float factor = __builtin_ldexpf(1.0f, -shift);
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t r = b16 * 16 + half * 8 + e;
      w[e] = *reinterpret_cast<const uint32_t*>(Q + min(r, (int64_t)rows - 1) * ld + min(k, (p.l.K - 1) & ~3));
    }
    const int keep = p.l.K - k;
    const uint32_t mask = keep <= 0 ? 0u : keep < 4 ? (1u << (8 * keep)) - 1 : 0xFFFFFFFFu;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = b16 * 16 + half * 8 + e < rows ? w[e] & mask : 0u;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __shfl(factor, (tid & 56) + e, 64);
    v4i* to = lds[wave] + (lane & ~7) * 4 + c4 * 4;        // (c ^ c4 / 4: two threads' 64 bytes are 256 apart)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v4i o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const v2f v = {(float)(int8_t)(w[2 * e] >> (8 * c)) * f[2 * e], (float)(int8_t)(w[2 * e + 1] >> (8 * c)) * f[2 * e + 1]};
        o[e] = __builtin_bit_cast(int, __builtin_convertvector(v, v2b));
      }
      to[c ^ (c4 >> 2)] = o;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (at0 + b < blocks) p.out[(at0 + b) * 64 + lane] = lds[wave][b * 64 + (lane ^ ((lane >> 4) & 1))];
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

struct WeightArgs {            // T of a piece
  LogitArgs l;
  const int64_t* targets;      // null: no row has a token
  const float *lse, *share, *given, *col;
  int v0, c0;                  // the first vocabulary row, and its place in the piece
  int tiles_v, tiles_t;        // of the piece
  int C16;                     // blocks of 16 vocabulary rows in a row of blocks
  int64_t first;               // tiles of the launch
  int count;
  int tb_log;                  // TB = 2^tb_log blocks of 32 tokens in a tile of dA's product
  v4i* T;                      // [tokens / (32 TB)][C16][TB][64]: the blocks that a stage of dA reads are in a row
  size_t plane;                // from a term of a value to the next (v4i)
};

// The forward tiles again, with T in place of the sums, written beside the next
// tile's loads: 8192 x 50304 x 768 in two terms 590 us for five pieces, 1.68 GB
// written; 2048 x 50257 x 768 in three terms 184 us for the wide tiles, 0.60 GB.
template <int TERMS, int BV, int BT, int WV, int WT, int PER_CU, int SB = 128, int S = 2>
__global__ void __launch_bounds__(WV * WT * 64, PER_CU * WV * WT / 4) head_weights_kernel(const WeightArgs p) {
  using Tile = LogitTile<BV, BT, WV, WT, SB, S>;
  constexpr int FV = Tile::FV, FT = Tile::FT;
  __shared__ __attribute__((aligned(1024))) int8_t smem[Tile::LDS];
  constexpr int TOKENS = Tile::TOKENS;
  __shared__ __attribute__((aligned(16))) float sc[2][BV], factor[2][BV];
  __shared__ float rows[2][4][TOKENS];                     // s_row, the log-sum-exp, share, given
  __shared__ int64_t targets[2][TOKENS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wv = wave / WT, wt = wave % WT;
  Walk walk((int)p.first, p.count, p.tiles_v * p.tiles_t);
  if (walk.at >= walk.end) return;
  int tv, tt;
  tile_of(walk.at, p.tiles_v, p.tiles_t, tv, tt);
  typename Tile::Source src;
  const auto start = [&](int turn) {
    const int t0 = tt * BT;
    Tile::template load_values<BV>(p.l.s_col, p.v0 + tv * BV, p.l.N, sc[turn]);
    Tile::template load_values<BV>(p.col, p.v0 + tv * BV, p.l.N, factor[turn]);
    Tile::template load_values<TOKENS>(p.l.s_row, t0, p.l.M, rows[turn][0]);
    Tile::template load_values<TOKENS>(p.lse, t0, p.l.M, rows[turn][1]);
    Tile::template load_values<TOKENS>(p.share, t0, p.l.M, rows[turn][2]);
    if (p.targets) {
      Tile::template load_values<TOKENS>(p.given, t0, p.l.M, rows[turn][3]);
      Tile::template load_values<2 * TOKENS>(p.targets, 2 * (int64_t)t0, 2 * (int64_t)p.l.M, targets[turn]);
    }
    Tile::start(p.l, smem, p.v0 + tv * BV, t0, src);
  };
  start(0);
  bool before = false;
  for (int turn = 0;; turn ^= 1) {
    const int v0 = p.v0 + tv * BV, t0 = tt * BT, tile_v = tv, tile_t = tt;
    v16i acc[FV][FT];
    // (a tile before this one left its T behind this one's first loads)
    Tile::template multiply<FT * FV * 2 * TERMS>(p.l, smem, src, before, acc);
    before = true;
    walk.at += walk.step;
    const bool more = walk.at < walk.end;
    if (more) {
      barrier_nofence();                                     // every wave has read this tile's last fragments
      tile_of(walk.at, p.tiles_v, p.tiles_t, tv, tt);
      start(turn ^ 1);
    }
    const float* col = sc[turn];
    const int half = lane >> 5;
    const bool ragged = v0 + BV > p.l.N;
#pragma unroll
    for (int j = 0; j < FT; ++j) {
      const int r = (wt * FT + j) * 32 + (lane & 31);
      // (no row, or one without a gradient: logits of 0 against an infinite lse, p = 0)
      float sr = 0.0f, share = 0.0f, given = 0.0f, lse2 = __builtin_inff();
      int target = -1024;                                    // in this tile, or far outside
      if (t0 + r < p.l.M) {
        const float lse = rows[turn][1][r];
        // a row whose log-sum-exp is off by a factor e or more in p has no gradient
        if (!(fabsf(lse) >= 16777216.0f)) {
          sr = rows[turn][0][r];
          lse2 = lse * kLog2e;
          const float rest = __builtin_fmaf(lse, kLog2e, -lse2);         // exp2(-rest) is the row's factor
          share = rows[turn][2][r] * __builtin_amdgcn_exp2f(-rest);
          if (p.targets) {
            const int64_t at = targets[turn][r];
            given = rows[turn][3][r];
            if (at >= v0 && at < v0 + BV && at < p.l.N) target = (int)(at - v0);
          }
        }
      }
      const int tb = tile_t * (BT / 32) + wt * FT + j;
      v4i* row = p.T + ((((size_t)(tb >> p.tb_log) * p.C16 + (size_t)(p.c0 / 16 + tile_v * (BV / 16))) << p.tb_log) + (tb & ((1 << p.tb_log) - 1))) * 64 + lane;
#pragma unroll
      for (int i = 0; i < FV; ++i) {
        const int r0 = (wv * FV + i) * 32 + 4 * half;
        float y[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v4f s4 = *reinterpret_cast<const v4f*>(col + r0 + 8 * q);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = epilogue1(acc[i][j][4 * q + e], sr, s4[e]);
            y[4 * q + e] = share * __builtin_amdgcn_exp2f(__builtin_fmaf(x, kLog2e, -lse2));
          }
        }
        const int in = target - r0;                       // 0 ... 27 for a row of this lane's
        if (__builtin_amdgcn_ballot_w64((unsigned)in < 28u) != 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (in == 8 * (e / 4) + e % 4) y[e] += given;
        }
        if (ragged) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (v0 + r0 + 8 * (e / 4) + e % 4 >= p.l.N) y[e] = 0.0f;
        }
        uint32_t w[TERMS][8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v4f s4 = *reinterpret_cast<const v4f*>(factor[turn] + r0 + 8 * q);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            v2f v = {y[4 * q + 2 * e] * s4[2 * e], y[4 * q + 2 * e + 1] * s4[2 * e + 1]};
#pragma unroll
            for (int term = 0; term < TERMS; ++term) {
              const v2b b = __builtin_convertvector(v, v2b);
              w[term][2 * q + e] = __builtin_bit_cast(uint32_t, b);
              const v2f back = __builtin_convertvector(b, v2f);
              v = v2f{v.x - back.x, v.y - back.y};         // exact
            }
          }
        }
        // lanes l and l ^ 32 hold rows 8q + 0..3 and 8q + 4..7: a fragment's lane
        // holds 8 in a row
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          v4i* to = row + ((size_t)((wv * FV + i) * 2 + s) << (p.tb_log + 6));
#pragma unroll
          for (int term = 0; term < TERMS; ++term) {
            const uint32_t* t = w[term];
            const auto a = __builtin_amdgcn_permlane32_swap(t[4 * s], t[4 * s + 2], false, false);
            const auto b = __builtin_amdgcn_permlane32_swap(t[4 * s + 1], t[4 * s + 3], false, false);
            to[term * p.plane] = v4i{(int)a[0], (int)b[0], (int)a[1], (int)b[1]};
          }
        }
      }
    }
    if (!more) return;
  }
}

// Both products of a piece.  A unit is a tile of 256 columns k (rows of the
// accumulators) by CT tokens (dA) or vocabulary rows (dBt), over a range of the
// contraction in stages of 32.
struct GradArgs {
  const v4i* T;
  size_t plane;                // from a term to the next (v4i)
  int C16;
  int KB, tiles_k;
  struct Side {
    const v4i* codes;          // [contraction / 16][KB][64]
    int tiles, splits;         // tiles of CT, ranges of the contraction
    int stages;                // of the whole contraction
    int per;                   // stages of a range
    float* planes;             // [splits][tiles][tiles_k][256 * CT] in register order, or null: write `out`
    int add;                   // add to the planes
    void* out;                 // the gradient's rows of the piece, `rows` of them exist
    int64_t ld;
    int rows;
    const Scale* scale;        // of its rows
  } a, b;                      // dA: contraction over the piece's vocabulary; dBt: over the tokens
  int units_a, units_b;
  int first;                   // place of the launch in every XCD's list
  int dtype, cols;
};

// How a tile is shared by the 8 waves.  FEW: at most 64 tokens, whose tile of
// dA is 64 wide, each wave 32 columns k of it; two workgroups run on a CU.
template <bool DUAL, bool FEW>
struct GradTile {
  static constexpr bool NARROW = FEW && !DUAL;
  static constexpr int WK = NARROW ? 8 : 2, WC = 8 / WK;   // waves along k and along CT
  static constexpr int FC = NARROW ? 2 : 1;                // 32-blocks of a wave along CT
  static constexpr int CT = 32 * FC * WC;
  static constexpr int FA = 8 / WK;                        // and along k: its i-th is block i WK + wk of the tile
  static constexpr int TB = FEW ? 2 : 4;                   // 32-token blocks of a tile of T
};

template <class T>
__device__ __forceinline__ void store4(T* to, int n, const float (&v)[4]) {
  T t[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) t[e] = from_f32<T>(v[e]);
  if (n >= 4) {
    __builtin_memcpy(to, t, sizeof(t));
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) to[e] = t[e];
  }
}
// Values k ... k + 3 of a gradient's row, n of them.
__device__ __forceinline__ void store_grad(void* out, int64_t ld, int dtype, int64_t row, int k, int n, v4f acc, Scale scale) {
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = scale.of(acc[e]);
  if (dtype == DT_F32) store4(static_cast<float*>(out) + row * ld + k, n, v);
  else if (dtype == DT_BF16) store4(static_cast<bf16_t*>(out) + row * ld + k, n, v);
  else store4(static_cast<f16_t*>(out) + row * ld + k, n, v);
}

// DUAL: dBt, for which T is read transposed.  A stage of 32 of the contraction
// is 16 KiB of codes and 8 of each term of T (4 for the narrow tile).  LDS holds five
// stages of two terms, and four of three: all but one are on their way while one is
// multiplied.  At most 64 tokens: three stages of dA of two terms and two of three,
// and dBt's two, in half of a CU's LDS.  FA: 32-blocks along k that a wave
// multiplies, fewer than the tile's where K ends in it.
constexpr int grad_stage(int terms, bool few, bool dual) { return 16384 + terms * (few && !dual ? 4096 : 8192); }
constexpr int grad_slots(int terms, bool few, bool dual) { return !few ? 7 - terms : dual ? 2 : 5 - terms; }
constexpr int grad_lds(int terms, bool few) {
  const int a = grad_stage(terms, few, false) * grad_slots(terms, few, false);
  const int b = grad_stage(terms, few, true) * grad_slots(terms, few, true);
  return a > b ? a : b;
}
static_assert(grad_lds(2, false) <= 163840 && grad_lds(3, false) <= 163840 && grad_lds(2, true) <= 81920 && grad_lds(3, true) <= 81920, "LDS");
template <int TERMS, bool DUAL, bool FEW, int FA>
__device__ __forceinline__ void grads_unit(const GradArgs& p, const GradArgs::Side& s, int u, int8_t* smem) {
  using Tile = GradTile<DUAL, FEW>;
  constexpr bool NARROW = Tile::NARROW;
  constexpr int kStage = grad_stage(TERMS, FEW, DUAL), kSlots = grad_slots(TERMS, FEW, DUAL);
  constexpr int WK = Tile::WK, WC = Tile::WC, FC = Tile::FC, CT = Tile::CT, TB = Tile::TB;
  constexpr int READS = FA + TERMS * FC * (DUAL ? 2 : 1), MFMAS = TERMS * FA * FC;   // of a k-step
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave / WC, wc = wave % WC;
  const int kt = u % p.tiles_k, ct = (u / p.tiles_k) % s.tiles, split = u / (p.tiles_k * s.tiles);
  const int first = split * s.per, n = min(s.per, s.stages - first);

  // sources of this wave's loads of a stage, two of codes and one to three of T: the
  // same in every lane but for the lane's 16 bytes of a block (codes behind KB are
  // not used: the last block in their place)
  constexpr int T_LOADS = NARROW ? TERMS - 1 : TERMS, LOADS = 2 + T_LOADS;
  const size_t row_a = (size_t)p.KB * 1024, row_b = (size_t)p.C16 * 1024, plane_b = p.plane * 16;
  const char* ga = reinterpret_cast<const char*>(s.codes) + (size_t)(first * 2) * row_a + (size_t)min(kt * 8 + wave, p.KB - 1) * 1024;
  const char* gb = reinterpret_cast<const char*>(p.T);
  const int lane_a = lane * 16;
  int lane_b = lane_a;
  if constexpr (NARROW) {
    // blocks [term][16 of the contraction 2][32 tokens 2]: 4 a term, two terms a load of all waves; the third
    // term's are loaded twice, to the same place
    gb += (size_t)(first * 2) * (TB * 1024) + (size_t)(wave & 3) * 1024;
  } else if constexpr (!DUAL) {
    // blocks [16 of the contraction 2][32 tokens TB], in a row; of each term 8
    gb += (size_t)ct * TB * row_b + (size_t)(first * 2) * (TB * 1024) + wave * 1024;
  } else {
    // 16 vocabulary rows each, of one block of 32 tokens; the 16-byte pieces of a block (half h, token t) are placed at
    // (h, t ^ (4h + 8 (vocabulary block % 2))), so that a transposing read of 32 lanes covers all banks
    lane_b = ((lane & 32) | ((lane & 31) ^ (4 * (lane >> 5) + 8 * (wave & 1)))) * 16;
    gb += ((size_t)ct * (CT / 16) + wave) * (TB * 1024);
  }
  auto issue = [&](int st) {
    int8_t* base = smem + (st % kSlots) * kStage;
    const char* a = ga + (size_t)st * 2 * row_a;
    const char* b = gb;
    if constexpr (!DUAL) {
      b += (size_t)st * (2 * TB * 1024);
    } else {
      const int tb = first + st;
      b += (size_t)(tb / TB) * (TB * row_b) + (size_t)(tb % TB) * 1024;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) lds_load16(a + q * row_a, lane_a, base + wave * 1024 + q * 8192);
#pragma unroll
    for (int q = 0; q < T_LOADS; ++q) {
      const int term = NARROW ? min(2 * q + (wave >> 2), TERMS - 1) : q;
      const int to = NARROW ? term * 4 + (wave & 3) : q * 8 + wave;
      lds_load16(b + term * plane_b, lane_b, base + 16384 + to * 1024);
    }
  };
  // LDS: codes [k-step 2][32 columns 8]; T [term][k-step 2][32 tokens TB], or [term][16 vocabulary rows CT / 16]
  constexpr int TERM = DUAL ? CT / 16 * 1024 : 2 * TB * 1024;
  const int offa = wk * 1024 + lane * 16;
  int offb, flip = 0;
  if constexpr (!DUAL) {
    offb = 16384 + wc * FC * 1024 + lane * 16;
  } else {
    const int g = lane >> 4, r = (lane & 15) >> 2, c = lane & 3, h = c >> 1;
    const int t = ((8 * (g >> 1)) ^ (8 * (g & 1))) + 4 * h + r;
    offb = 16384 + (wc * FC * 2 + (g & 1)) * 1024 + h * 512 + t * 16 + (c & 1) * 8;
    flip = offb ^ 64;                                       // the fragment's other 4 tokens
  }
  v16f acc[FA][FC];
  // register order of a plane: [wave][i][j][q][lane] of 4 values
  float* plane = s.planes ? s.planes + ((size_t)(split * s.tiles + ct) * p.tiles_k + kt) * (256 * CT) + (size_t)wave * (Tile::FA * FC * 1024) + lane * 4
                          : nullptr;
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FC; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  auto read = [&](const int8_t* base, auto ks_t, v8b (&fa)[FA], v8b (&fb)[TERMS][FC]) {
    constexpr int ks = decltype(ks_t)::value;
#pragma unroll
    for (int i = 0; i < FA; ++i) fa[i] = *reinterpret_cast<const v8b*>(base + offa + ks * 8192 + i * (WK * 1024));
#pragma unroll
    for (int t = 0; t < TERMS; ++t)
#pragma unroll
      for (int j = 0; j < FC; ++j) {
        if constexpr (!DUAL) {
          fb[t][j] = *reinterpret_cast<const v8b*>(base + offb + t * TERM + ks * (TB * 1024) + j * 1024);
        } else {
          // tokens 16 ks ... of the block
          const int at = t * TERM + j * 2048 + ks * 256;
          typedef __attribute__((address_space(3))) v4s lds_v4s;
          const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(base + offb + at));
          const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(base + flip + at));
          union { v4s h[2]; v8b v; } f{{x, y}};
          fb[t][j] = f.v;
        }
      }
  };
  auto mfma = [&](const v8b (&fa)[FA], const v8b (&fb)[TERMS][FC]) {
#pragma unroll
    for (int t = 0; t < TERMS; ++t)
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FC; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[t][j], acc[i][j], 0, 0, 0);
  };
  const std::integral_constant<int, 0> k0;
  const std::integral_constant<int, 1> k1;
  v8b fa0[FA], fa1[FA], fb0[TERMS][FC], fb1[TERMS][FC];
  if constexpr (FEW && DUAL) {
    // 64 tokens are two stages
    issue(0);
    if (n > 1) issue(1);
    wait_loads<0>();
    barrier_nofence();
    for (int st = 0; st < n; ++st) {
      read(smem + st * kStage, k0, fa0, fb0);
      read(smem + st * kStage, k1, fa1, fb1);
      mfma(fa0, fb0);
      mfma(fa1, fb1);
    }
  } else {
    // n is 8 at least: contractions are whole blocks of 256
#pragma unroll
    for (int st = 0; st < kSlots; ++st) issue(st);
    wait_loads<LOADS * (kSlots - 1)>();
    barrier_nofence();
    read(smem, k0, fa0, fb0);
    int slot = 0;
    // one stage; the next one's first fragments are read behind the barrier that
    // frees this one's slot, and multiplied after it
    auto stage = [&](int st, auto left_t) {                // left: stages in flight behind the next one
      constexpr int left = decltype(left_t)::value;
      const int8_t* base = smem + slot * kStage;
      slot = slot + 1 == kSlots ? 0 : slot + 1;
      read(base, k1, fa1, fb1);
      mfma(fa0, fb0);
      interleave<READS, MFMAS>();
      // the next stage has landed, and this one's last fragments are in registers
      wait_loads<LOADS * left>();
      barrier_nofence();
      if constexpr (left == kSlots - 2) {
        if (st + kSlots < n) issue(st + kSlots);
      }
      read(smem + slot * kStage, k0, fa0, fb0);
      mfma(fa1, fb1);
      interleave<READS, MFMAS>();
    };
    int st = 0;
    for (; st + kSlots - 1 < n; ++st) stage(st, std::integral_constant<int, kSlots - 2>{});
    if constexpr (kSlots > 4) stage(st++, std::integral_constant<int, 2>{});
    if constexpr (kSlots > 3) stage(st++, std::integral_constant<int, 1>{});
    if constexpr (kSlots > 2) stage(st, std::integral_constant<int, 0>{});
    read(smem + slot * kStage, k1, fa1, fb1);
    mfma(fa0, fb0);
    interleave<READS, MFMAS>();
    mfma(fa1, fb1);
  }

  if (plane) {
    // (what is added to is read before the stores of two rows of blocks: a load
    // behind a store would wait for it)
    constexpr int STEP = FA < 2 ? 1 : 2;
#pragma unroll
    for (int i0 = 0; i0 < FA; i0 += STEP) {
      v4f old[STEP][FC][4];
      if (s.add) {
#pragma unroll
        for (int i = 0; i < STEP; ++i)
#pragma unroll
          for (int j = 0; j < FC; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) old[i][j][q] = *reinterpret_cast<const v4f*>(plane + (((i0 + i) * FC + j) * 4 + q) * 256);
      }
#pragma unroll
      for (int i = 0; i < STEP; ++i)
#pragma unroll
        for (int j = 0; j < FC; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const v16f& a = acc[i0 + i][j];
            v4f v = {a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
            if (s.add) v += old[i][j][q];
            *reinterpret_cast<v4f*>(plane + (((i0 + i) * FC + j) * 4 + q) * 256) = v;
          }
    }
    return;
  }
  const auto write = [&](auto type) {
    using T = decltype(type);
    constexpr int ROW = 256 * sizeof(T) + 16;              // (the 16 spread a column's values over the banks)
    constexpr int COLS = grad_lds(TERMS, FEW) / ROW >= CT ? CT : CT / 2, N = 16 / sizeof(T), LANES = 256 / N;
    static_assert(COLS * ROW <= grad_lds(TERMS, FEW) && COLS % (32 * FC) == 0, "whole waves' columns at a time");
#pragma unroll
    for (int c0 = 0; c0 < CT; c0 += COLS) {
      __syncthreads();
      if (wc * FC * 32 >= c0 && wc * FC * 32 < c0 + COLS) {
#pragma unroll
        for (int j = 0; j < FC; ++j) {
          const int in = (wc * FC + j) * 32 + (lane & 31), col = ct * CT + in;
          const Scale scale = col < s.rows ? s.scale[col] : Scale{0.0f, 0};
          int8_t* to = smem + (in - c0) * ROW + 4 * (lane >> 5) * sizeof(T);
#pragma unroll
          for (int i = 0; i < FA; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              T v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = from_f32<T>(scale.of(acc[i][j][4 * q + e]));
              __builtin_memcpy(__builtin_assume_aligned(to + ((i * WK + wk) * 32 + 8 * q) * sizeof(T), 4 * sizeof(T)), v, sizeof(v));
            }
        }
      }
      __syncthreads();
      const int k = kt * 256 + lane % LANES * N, n = p.cols - k;
      for (int r = wave * (64 / LANES) + lane / LANES; r < COLS; r += 8 * (64 / LANES)) {
        const int col = ct * CT + c0 + r;
        if (col >= s.rows || n <= 0) continue;
        const v4i x = *reinterpret_cast<const v4i*>(smem + r * ROW + lane % LANES * 16);
        T* to = static_cast<T*>(s.out) + col * s.ld + k;
        if (n >= N) {
          __builtin_memcpy(to, &x, 16);
        } else {
          T v[N];
          __builtin_memcpy(v, &x, 16);
#pragma unroll
          for (int e = 0; e < N - 1; ++e)
            if (e < n) to[e] = v[e];
        }
      }
    }
  };
  // A tile's rows through LDS: a store has 512 bytes of a row or more (23 x 12669 x
  // 1716 bf16, products of one term, 63 us, and 95 where a lane stores its 8 bytes of
  // 32 rows).
  if (TERMS == 2) write(bf16_t{});
  else if (p.dtype == DT_F32) write(float{});
  else write(f16_t{});
}

// Each XCD (workgroups are dealt to the 8 in turn) takes an eighth of either
// side's units, neighbours in their order: they share T or codes in its L2.
// The longer ones go first.  8192 x 50304 x 768 bf16, two terms: 2.53 TFLOP in
// five launches of 463 us (medians), 1.09 PFLOPS (library products of these shapes
// reach 0.82 and 1.05); 2048 x 50257 x 768 f32, three terms: 0.95 TFLOP in 764 us,
// 1.24 PFLOPS.  The matrix cores are busy 64 and 68% of the time, at 1.8 to 1.9 GHz.
// (Dealt without regard to the XCDs, dA's units came to lie on one: the latter, with
// two terms, took 1783 us in all, and 791 as they are dealt here.)
// LAST: 32-blocks along k that a wave multiplies in the last tile of k.
template <int TERMS, bool FEW, int LAST>
__global__ void __launch_bounds__(512, FEW ? 4 : 2) head_grads_kernel(const GradArgs p) {
  __shared__ __attribute__((aligned(1024))) int8_t smem[grad_lds(TERMS, FEW)];
  const int xcd = blockIdx.x & 7, at = p.first + (blockIdx.x >> 3);
  const int a0 = (int)((int64_t)p.units_a * xcd / 8), na = (int)((int64_t)p.units_a * (xcd + 1) / 8) - a0;
  const int b0 = (int)((int64_t)p.units_b * xcd / 8), nb = (int)((int64_t)p.units_b * (xcd + 1) / 8) - b0;
  const bool a_first = p.a.per >= p.b.per;
  const int n1 = a_first ? na : nb;
  if (at >= na + nb) return;
  const bool second = at >= n1;
  const int in = second ? at - n1 : at;
  if (a_first != second) {
    const int u = a0 + in;
    if constexpr (FEW) grads_unit<TERMS, false, true, 1>(p, p.a, u, smem);
    else if (LAST == 4 || u % p.tiles_k + 1 < p.tiles_k) grads_unit<TERMS, false, false, 4>(p, p.a, u, smem);
    else grads_unit<TERMS, false, false, LAST>(p, p.a, u, smem);
  } else {
    const int u = b0 + in;
    if (LAST == 4 || u % p.tiles_k + 1 < p.tiles_k) grads_unit<TERMS, true, FEW, 4>(p, p.b, u, smem);
    else grads_unit<TERMS, true, FEW, LAST>(p, p.b, u, smem);
  }
}

struct FinishArgs {
  struct Side {
    const float* planes;
    int splits, tiles;
    int CT, WK;                // of the tile
    void* out;
    int64_t ld;
    int rows;
    const Scale* scale;
  } side[2];
  int64_t groups;              // workgroups of side[0]; those behind take side[1]
  int tiles_k, dtype, cols;
};
// The planes' sum, in their order, by its row's scale: memory, 8192 x 768 with 4
// planes 28 us for 114 MB.
__global__ void __launch_bounds__(256) head_finish_kernel(const FinishArgs p) {
  const bool second = blockIdx.x >= p.groups;
  const FinishArgs::Side& s = p.side[second];
  const int64_t group = second ? blockIdx.x - p.groups : blockIdx.x, groups = second ? gridDim.x - p.groups : p.groups;
  const size_t size = (size_t)256 * s.CT, all = (size_t)s.tiles * p.tiles_k * size;
  const int WC = 8 / s.WK, FC = s.CT / 32 / WC, FA = 8 / s.WK;
  for (size_t at = ((size_t)group * 256 + threadIdx.x) * 4; at < all; at += (size_t)groups * 1024) {
    const int tile = (int)(at / size), in = (int)(at % size) / 4;
    const int kt = tile % p.tiles_k, ct = tile / p.tiles_k;
    const int lane = in & 63, q = (in >> 6) & 3, j = (in >> 8) % FC, i = (in >> 8) / FC % FA, wave = (in >> 8) / (FC * FA);
    const int col = ct * s.CT + (wave % WC * FC + j) * 32 + (lane & 31);
    const int k = kt * 256 + (i * s.WK + wave / WC) * 32 + 8 * q + 4 * (lane >> 5);
    if (col >= s.rows || k >= p.cols) continue;
    v4f v = *reinterpret_cast<const v4f*>(s.planes + at);
#pragma unroll 8
    for (int n = 1; n < s.splits; ++n) v += *reinterpret_cast<const v4f*>(s.planes + n * all + at);
    store_grad(s.out, s.ld, p.dtype, col, k, p.cols - k, v, s.scale[col]);
  }
}

// The gradient of no tokens.
__global__ void __launch_bounds__(256) head_zero_kernel(void* out, int64_t ld, int dtype, int64_t rows, int cols) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int k = threadIdx.x * 4; k < cols; k += 1024) store_grad(out, ld, dtype, r, k, cols - k, v4f{0, 0, 0, 0}, Scale{1.0f, 0});
}

constexpr int64_t kMostGroups = int64_t(1) << 22;   // workgroups of a launch

int up(int64_t a, int b) { return (int)((a + b - 1) / b); }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

LogitArgs logit_args(const HeadArgs& a) {
  return LogitArgs{a.A, a.B, a.s_row, a.s_col, a.lda, a.ldb, (int)a.M, (int)a.N, (int)a.K};
}

// Tiles of logits: 256 vocabulary rows by 256 tokens, or, with three workgroups a
// CU, 128 by 64 or 128 by 32, which leave more of the chip busy where there are
// few, and fewer tokens unused.  The times (us) of a round of 256 or 768 of them
// are fitted to 13 shapes: 8192 x 16384 x 768 takes 145, 178 and 242 us, 1180 x
// 13260 x 246 29.3, 22.7 and 26.9, one token x 50257 x 768 21.3, 13.9 and 13.0.
// Wide tiles may take whole rounds of the vocabulary's first columns and the
// small ones the rest, in a launch of their own.
struct LogitPlan {
  int64_t wide;                // columns of the wide tiles (whole tiles, or all)
  int bv, bt;                  // of the others
  double time;
};
LogitPlan logit_plan(int64_t M, int64_t N, int64_t K) {
  const double k = (double)((K + 127) / 128), round = 6.0 + 1.7 * k;
  const auto small = [&](int64_t n) {
    const auto of = [&](int bt, double t) {
      const double tiles = (double)((n + 127) / 128) * (double)((M + bt - 1) / bt) / 768;
      return (tiles < 0.6 ? 0.6 : tiles) * t;
    };
    const double mid = of(64, 2.4 + 1.0 * k), thin = of(32, 1.7 + 0.7 * k);
    return thin < mid ? LogitPlan{0, 128, 32, thin} : LogitPlan{0, 128, 64, mid};
  };
  const int64_t across = (M + 255) / 256, all = (N + 255) / 256, rounds = all * across / 256;
  const LogitPlan wide{N, 128, 64, (double)((all * across + 255) / 256) * round};
  LogitPlan best = small(N);
  if (wide.time < best.time) best = wide;
  const int64_t cols = rounds * 256 / across;              // tile columns of whole rounds
  if (cols > 0 && cols < all) {
    LogitPlan part = small(N - cols * 256);
    part.time += (double)((cols * across + 255) / 256) * round + 3.0;
    part.wide = cols * 256;
    if (part.time < best.time) best = part;
  }
  return best;
}

// Wide tiles in four stages of 64 bytes of K where they multiply fewer zeros behind
// K than two of 128 do: 8192 x 8192 x 64 38.6 us and 45.2, 2048 x 50257 x 300 87.7
// and 92.5, 4096 x 50304 x 1600 362 and 368; but 8192 x 50304 x 768 385 and 363.
bool short_stages(int64_t K) { return K > 0 && (K - 1) % 128 < 64; }

// Workgroups of a launch over tiles: at most one a CU for the wide ones, each of
// which walks over several.
dim3 tile_grid(int64_t tiles, bool wide) {
  const int64_t n = (tiles + 7) / 8 * 8;
  return dim3((unsigned)(wide && n > 256 ? 256 : n));
}

// Tokens of a launch, which bounds its workspace and grid (vocabulary rows are
// at most 2^22, so tiles at most 2^22).
constexpr int64_t kFwdRows = 65536;

// Pieces of the vocabulary and, in each, the ranges that the products'
// contractions are split into: a piece's T has at most piece_bytes (or 256 columns);
// among the allowed the least estimated time is taken.
constexpr int64_t piece_bytes(int terms) { return int64_t(3) << (25 + terms); }   // 403 MB, 805 MB
struct BwdPlan {
  int terms;
  bool few;                    // at most 64 tokens
  int ca, cb, tb_log;          // CT of dA's and dBt's tiles, and TB, as GradTile has them
  int64_t Mp, C;
  int pieces, tiles_k, sa, sb;
  int KB;                      // 32-blocks of K, in pairs
  size_t code_a, code_b, t, plane_a, plane_b;   // bytes
  size_t rows, cols;           // what is kept of tokens and of vocabulary rows, in whole 256s
  size_t bytes() const { return kBounds * sizeof(Bound) + rows * 16 + cols * 12 + code_a + code_b + t + plane_a + plane_b; }
};
// When units of two lengths are done on the 32 CUs of an XCD, which takes an
// eighth of them: the longer ones first, then each CU the next one as it
// becomes free.
double makespan(int64_t n1, double t1, int64_t n2, double t2) {
  if (t1 < t2) {
    std::swap(n1, n2);
    std::swap(t1, t2);
  }
  n1 = (n1 + 7) / 8;
  n2 = (n2 + 7) / 8;
  const int64_t late = n1 % 32, soon = 32 - late;          // CUs that end the longer ones at `low` and at `high`
  const double low = (double)(n1 / 32) * t1, high = low + t1;
  if (n2 == 0) return late ? high : low;
  const int64_t lag = (int64_t)(t1 / t2);                  // whole short units between the two
  double end = 1e300;
  // the earliest end of a short unit by which all of them fit
  for (int64_t k = n2 / 32 > 1 ? n2 / 32 - 1 : 1; end == 1e300; ++k)      // ends of CUs that started at `low`
    if (soon * k + late * (k > lag ? (int64_t)(((double)k * t2 - t1) / t2) : 0) >= n2) end = low + (double)k * t2;
  if (late == 0) return end;
  for (int64_t k = 0;; ++k) {                              // and at `high`
    const double t = high + (double)k * t2;
    if (t >= end) break;
    if (soon * (int64_t)((t - low) / t2) + late * k >= n2) end = t;
  }
  return end > high ? end : high;
}
BwdPlan bwd_plan(int64_t M, int64_t N, int64_t K, int dtype) {
  BwdPlan b;
  b.terms = dtype == DT_BF16 ? 2 : 3;
  b.few = M <= 64;
  b.cb = 128;
  b.ca = b.few ? 64 : 128;
  b.tb_log = b.few ? 1 : 2;
  b.Mp = b.few ? 64 : (M + 255) / 256 * 256;
  b.tiles_k = up(K, 256);
  const int64_t blocks = (N + 255) / 256;                  // of 256 columns
  int64_t most = piece_bytes(b.terms) / (b.Mp * 512 * b.terms);
  if (most < 1) most = 1;
  const int64_t least = (blocks + most - 1) / most;
  const int64_t ta = b.Mp / b.ca * b.tiles_k, db = up(b.Mp, 256);
  // microseconds, fitted to 25 plans at 8192 x 50304 x 768 (bf16) and 2048 x
  // 50257 x 768 (f32) with products of as many terms, whose times it orders as they
  // are to a few per cent: 64 of the contraction of a unit, a term's half of 1.65; a
  // unit's start and end, two launches; planes at 4 TB/s
  const double kStep = 0.825 * b.terms;
  constexpr double kUnit = 6.0, kLaunches = 8.0;
  double best = 1e300;
  b.sa = b.sb = b.pieces = 1;
  b.C = 256;
  for (int64_t pieces = least; pieces <= least + 3 && pieces <= blocks; ++pieces) {
    const int64_t c = (blocks + pieces - 1) / pieces, n = (blocks + c - 1) / c, last = blocks - (n - 1) * c;
    const double weights = logit_plan(b.Mp, c * 256, K).time;
    for (int64_t sa = 1; sa <= 64 && sa <= c; sa += sa < 4 ? 1 : sa)
      for (int64_t sb = 1; sb <= 64 && sb <= db; sb += sb < 4 ? 1 : sb) {
        const int64_t pa = (c + sa - 1) / sa, pb = (db + sb - 1) / sb;
        const double ua = kUnit + kStep * 4 * (double)pa, ub = kUnit + kStep * 4 * (double)pb;
        const int64_t na = ta * ((c + pa - 1) / pa), nb = 256 / b.cb * b.tiles_k * ((db + pb - 1) / pb);   // nb: for 256 columns
        const double planes = (double)(b.Mp * b.tiles_k) * 1024 * sa * 2 * n + (sb > 1 ? (double)(blocks * 256 * b.tiles_k) * 1024 * sb * 2 : 0.0);
        const double t = n * (weights + kLaunches + (sb > 1 ? 4.0 : 0.0)) + (n - 1) * makespan(na, ua, nb * c, ub) +
                         makespan(na, ua, nb * last, ub) + planes / 4e6;
        if (t < best) {
          best = t;
          b.sa = (int)sa;
          b.sb = (int)sb;
          b.pieces = (int)n;
          b.C = c * 256;
        }
      }
  }
  b.rows = align256((size_t)M);
  b.cols = align256((size_t)N);
  b.KB = up(K, 64) * 2;
  b.code_a = (size_t)b.Mp * b.KB * 64;
  b.code_b = (size_t)b.C * b.pieces * b.KB * 64;
  b.t = (size_t)b.Mp * b.C * 2 * b.terms;
  b.plane_a = b.sa > 1 || b.pieces > 1 ? (size_t)b.Mp * b.tiles_k * 1024 * b.sa : 0;
  b.plane_b = b.sb > 1 ? (size_t)b.C * b.tiles_k * 1024 * b.sb : 0;
  return b;
}

}  // namespace

template <int TERMS, bool FEW>
static void launch_grads_of(int last, unsigned n, hipStream_t stream, const GradArgs& p) {
  if (last > 2) hipLaunchKernelGGL((head_grads_kernel<TERMS, FEW, 4>), dim3(n), dim3(512), 0, stream, p);
  else if (last == 2) hipLaunchKernelGGL((head_grads_kernel<TERMS, FEW, 2>), dim3(n), dim3(512), 0, stream, p);
  else hipLaunchKernelGGL((head_grads_kernel<TERMS, FEW, 1>), dim3(n), dim3(512), 0, stream, p);
}
static void launch_grads(const BwdPlan& b, int K, unsigned n, hipStream_t stream, const GradArgs& p) {
  const int last = (K - (b.tiles_k - 1) * 256 + 63) / 64;  // pairs of 32 columns in the last tile
  if (b.terms == 2 && b.few) launch_grads_of<2, true>(last, n, stream, p);
  else if (b.terms == 2) launch_grads_of<2, false>(last, n, stream, p);
  else if (b.few) launch_grads_of<3, true>(last, n, stream, p);
  else launch_grads_of<3, false>(last, n, stream, p);
}

size_t head_fwd_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t rows = M < kFwdRows ? M : kFwdRows;
  const LogitPlan pl = logit_plan(rows, N, K);
  return align256((size_t)(up(pl.wide, 256) + up(N - pl.wide, 128)) * (size_t)rows * sizeof(v2f));
}

hipError_t launch_head_fwd(const HeadArgs& whole, const int64_t* targets, float* logprob, float* lse, void* ws, hipStream_t stream) {
  const LogitPlan pl = logit_plan(whole.M < kFwdRows ? whole.M : kFwdRows, whole.N, whole.K);
  for (int64_t row = 0; row < whole.M; row += kFwdRows) {
    HeadArgs a = whole;
    a.M = whole.M - row < kFwdRows ? whole.M - row : kFwdRows;
    a.A += row * a.lda;
    a.s_row += row;
    FwdArgs f{logit_args(a), 0, up(pl.wide, 256), up(a.M, 256), static_cast<v2f*>(ws)};
    if (f.tiles_v > 0) {
      const dim3 grid = tile_grid((int64_t)f.tiles_v * f.tiles_t, true);
      if (short_stages(a.K)) hipLaunchKernelGGL((head_fwd_kernel<256, 256, 2, 4, 1, 64, 4>), grid, dim3(512), 0, stream, f);
      else hipLaunchKernelGGL((head_fwd_kernel<256, 256, 2, 4, 1>), grid, dim3(512), 0, stream, f);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    int n_parts = f.tiles_v;
    if (pl.wide < a.N) {
      f.v0 = (int)pl.wide;
      f.parts += (size_t)n_parts * a.M;
      f.tiles_v = up(a.N - pl.wide, pl.bv);
      f.tiles_t = up(a.M, pl.bt);
      n_parts += f.tiles_v;
      const dim3 grid = tile_grid((int64_t)f.tiles_v * f.tiles_t, false);
      if (pl.bt == 32) hipLaunchKernelGGL((head_fwd_kernel<128, 32, 4, 1, 3>), grid, dim3(256), 0, stream, f);
      else hipLaunchKernelGGL((head_fwd_kernel<128, 64, 4, 1, 3>), grid, dim3(256), 0, stream, f);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    JoinArgs j{f.l, targets ? targets + row : nullptr, static_cast<const v2f*>(ws), n_parts, logprob ? logprob + row : nullptr, lse ? lse + row : nullptr};
    if (a.M >= 1024) hipLaunchKernelGGL(head_join_kernel<16>, dim3((unsigned)up(a.M, 16)), dim3(256), 0, stream, j);
    else hipLaunchKernelGGL(head_join_kernel<1>, dim3((unsigned)a.M), dim3(256), 0, stream, j);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

size_t head_bwd_bytes(int64_t M, int64_t N, int64_t K, int dtype) { return bwd_plan(M, N, K, dtype).bytes(); }

hipError_t launch_head_bwd(const HeadArgs& a, const HeadGradArgs& g, void* ws, hipStream_t stream) {
  if (a.M == 0) {
    hipLaunchKernelGGL(head_zero_kernel, dim3((unsigned)(a.N < 65536 ? a.N : 65536)), dim3(256), 0, stream, g.dB, g.lddb, g.dtype,
                       a.N, (int)a.K);
    return hipGetLastError();
  }
  const BwdPlan b = bwd_plan(a.M, a.N, a.K, g.dtype);
  char* at = static_cast<char*>(ws);
  Bound* bounds = reinterpret_cast<Bound*>(at);
  Scale* scale_a = reinterpret_cast<Scale*>(at += kBounds * sizeof(Bound));
  Scale* scale_b = scale_a + b.rows;
  float* share = reinterpret_cast<float*>(scale_b + b.cols);
  float *given = share + b.rows, *col = given + b.rows;
  v4i* code_a = reinterpret_cast<v4i*>(at += b.rows * 16 + b.cols * 12);
  v4i* code_b = reinterpret_cast<v4i*>(at += b.code_a);
  v4i* T = reinterpret_cast<v4i*>(at += b.code_b);
  float* plane_a = reinterpret_cast<float*>(at += b.t);
  float* plane_b = reinterpret_cast<float*>(at += b.plane_a);
  const int KB = b.KB;
  const int C16 = (int)(b.C / 16);
  const size_t plane = (size_t)b.Mp * b.C / 8;
  const LogitArgs l = logit_args(a);
  const int64_t* targets = g.g_logprob ? g.targets : nullptr;
  const RowArgs rows{targets, g.g_logprob, g.g_lse, a.s_row, a.s_col, (int)a.M, (int)a.N};
  const bool own = a.M + a.N <= kOwnBounds;
  if (!own) hipLaunchKernelGGL(head_bounds_kernel, dim3(kBounds), dim3(256), 0, stream, rows, bounds);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  PackArgs k{l,      rows,   own ? nullptr : bounds, (int)(b.Mp / 16), (int)(b.C * b.pieces / 16), KB, code_a, share, given, col,
             scale_a, scale_b};
  const int64_t groups = ((int64_t)(k.blocks_a + (int64_t)k.blocks_b) * KB + 15) / 16;
  hipLaunchKernelGGL(head_prepare_kernel, dim3((unsigned)(groups < kMostGroups ? groups : kMostGroups)), dim3(256), 0, stream, k);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const auto finish_side = [&](bool a_side, const GradArgs::Side& s) {
    return FinishArgs::Side{s.planes, s.splits, s.tiles, a_side ? b.ca : b.cb, a_side && b.few ? 8 : 2, s.out, s.ld, s.rows, s.scale};
  };
  for (int piece = 0; piece < b.pieces; ++piece) {
    const int64_t v0 = piece * b.C, n_rows = a.N - v0 < b.C ? a.N - v0 : b.C;
    WeightArgs w{l, targets, g.lse, share, given, col, (int)v0, 0, 0, 0, C16, 0, 0, b.tb_log, T, plane};
    const LogitPlan pl = logit_plan(b.Mp, b.C, a.K);
    const int64_t wide_cols = b.few ? 0 : pl.wide;         // (few tokens: T has 64)
    for (const bool wide : {true, false}) {
      w.c0 = wide ? 0 : (int)wide_cols;
      w.v0 = (int)v0 + w.c0;
      w.tiles_v = (int)(wide ? wide_cols / 256 : (b.C - wide_cols) / 128);
      w.tiles_t = (int)(b.Mp / (wide ? 256 : 64));
      for (w.first = 0; w.first < (int64_t)w.tiles_v * w.tiles_t; w.first += kMostGroups) {
        const int64_t left = (int64_t)w.tiles_v * w.tiles_t - w.first;
        w.count = (int)(left < kMostGroups ? left : kMostGroups);
        const dim3 grid = tile_grid(w.count, wide);
        const bool brief = short_stages(a.K);
        if (wide && b.terms == 2 && brief) hipLaunchKernelGGL((head_weights_kernel<2, 256, 256, 2, 4, 1, 64, 4>), grid, dim3(512), 0, stream, w);
        else if (wide && brief) hipLaunchKernelGGL((head_weights_kernel<3, 256, 256, 2, 4, 1, 64, 4>), grid, dim3(512), 0, stream, w);
        else if (wide && b.terms == 2) hipLaunchKernelGGL((head_weights_kernel<2, 256, 256, 2, 4, 1>), grid, dim3(512), 0, stream, w);
        else if (wide) hipLaunchKernelGGL((head_weights_kernel<3, 256, 256, 2, 4, 1>), grid, dim3(512), 0, stream, w);
        else if (b.terms == 2) hipLaunchKernelGGL((head_weights_kernel<2, 128, 64, 4, 1, 3>), grid, dim3(256), 0, stream, w);
        else hipLaunchKernelGGL((head_weights_kernel<3, 128, 64, 4, 1, 3>), grid, dim3(256), 0, stream, w);
        if ((e = hipGetLastError()) != hipSuccess) return e;
      }
    }

    GradArgs p{};
    p.T = T;
    p.plane = plane;
    p.C16 = C16;
    p.KB = KB;
    p.tiles_k = b.tiles_k;
    p.dtype = g.dtype;
    p.cols = (int)a.K;
    const auto side = [](const v4i* codes, int64_t tiles, int64_t depth, int splits, float* planes, int add, void* out, int64_t ld,
                         int64_t n, const Scale* scale) {
      // (whole blocks of 256: a range has 8 stages at least; 64 tokens are 2)
      const int stages = (int)(depth / 32), per = stages < 8 ? stages : up(stages / 8, splits) * 8;
      return GradArgs::Side{codes, (int)tiles, up(stages, per), stages, per, planes, add, out, ld, (int)n, scale};
    };
    const int64_t esize = g.dtype == DT_F32 ? 4 : 2;
    p.a = side(code_b + (size_t)piece * (b.C / 16) * KB * 64, b.Mp / b.ca, b.C, b.sa, b.plane_a > 0 ? plane_a : nullptr, piece > 0, g.dA,
               g.ldda, a.M, scale_a);
    p.b = side(code_a, up(n_rows, b.cb), b.Mp, b.sb, b.sb > 1 ? plane_b : nullptr, 0,
               g.dB ? static_cast<char*>(g.dB) + v0 * g.lddb * esize : nullptr, g.lddb, n_rows, scale_b + v0);
    p.units_a = g.dA ? p.tiles_k * p.a.tiles * p.a.splits : 0;
    p.units_b = g.dB ? p.tiles_k * p.b.tiles * p.b.splits : 0;
    const int most = up(p.units_a, 8) + up(p.units_b, 8);    // of an XCD
    for (p.first = 0; p.first < most; p.first += kMostGroups / 8) {
      const unsigned n = 8u * (unsigned)(most - p.first < kMostGroups / 8 ? most - p.first : kMostGroups / 8);
      launch_grads(b, (int)a.K, n, stream, p);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    FinishArgs f{};
    f.tiles_k = b.tiles_k;
    f.dtype = g.dtype;
    f.cols = (int)a.K;
    int64_t finish_groups[2] = {0, 0};
    int n = 0;
    const auto take = [&](bool a_side, const GradArgs::Side& s) {
      f.side[n] = finish_side(a_side, s);
      const int64_t all = (int64_t)s.tiles * b.tiles_k * (a_side ? b.ca : b.cb) / 4;
      finish_groups[n++] = all < kMostGroups ? all : kMostGroups;
    };
    if (g.dA && p.a.planes && piece + 1 == b.pieces) take(true, p.a);
    if (g.dB && p.b.planes) take(false, p.b);
    f.groups = finish_groups[0];
    if (n > 0) hipLaunchKernelGGL(head_finish_kernel, dim3((unsigned)(finish_groups[0] + finish_groups[1])), dim3(256), 0, stream, f);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace i8g
