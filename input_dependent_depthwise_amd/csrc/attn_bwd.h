// attn_bwd.h -- causal attention over whole sequences, backward: the kernels
// (compiled by attn_bwd_bf16.hip and attn_bwd_fp32.hip, and with a window by attn_window_bwd_bf16.hip
// and attn_window_bwd_fp32.hip).
//
// Two kernels, neither with atomics: dq with queries owned by the lanes and
// keys streamed (it also forms delta = do . o), then dk and dv with keys owned
// and queries streamed.  The scores are formed twice (7 products where 5 would
// do), which costs less than a fixed-order sum of dq over blocks of keys.
//
// Bound by the matrix cores and the vector units: 16 + 4 heads of 128, 8192 tokens, bf16: dq 406 us
// (3 products, 1.01 PFLOP/s), dk/dv 621 us (4 products, 0.89 PFLOP/s).  dq has two waves on a
// SIMD (three with heads of 64).  dk/dv holds a key's and a value's row and both of their sums,
// over 256 registers with heads of 128, so one wave has a SIMD for itself and its products are
// put in an order that fills the gaps by hand.
//
// Through a window a key is seen by as many queries; sinks are seen by all that follow, which would be one block's
// work: attn_far_kernel sums them for the queries past the window and dk/dv adds its sums.  16 + 4 heads of 128, 8192 tokens in
// 2 documents, window of 1024, 4 sinks, bf16: forward 96 to 102 with the card, dq 130 to 138, sinks 19, dk/dv 240 to 247 us (matrix
// cores 36 % busy in dq, 29 % in dk/dv); 12 heads of 64, 8 rows of 2048, window of 256: 45, 62, 14, 76.
#pragma once

#include <type_traits>

#include "attn.h"
#include "kernels.h"

namespace dynconv {

namespace {

template <typename T, int DH, int BN, bool REST, bool WIN>
struct Dq {
  using TL = Tile<T, DH>;
  typedef unsigned char Lds[2][2][TL::bytes(BN)];  // [buffer][key, value]
  // the block: keys of its head, their range, valid tokens
  const char *kh, *vh;
  int64_t krow, vrow;
  int first, last, limit, hd;
  // the wave: its first query, first key, and the key from which on every row sees keys
  int qw, w_first, w_full;
  int q, start;  // the lane's query and its document's start
  Window<BN, WIN> win;
  static constexpr bool STAGED = WIN;  // (as in the forward, here for the keys)
  float c;       // scale log2 e
  float lse2, delta;
  uint4 qf[TL::KS], df[TL::KS];
  f32x16 acc[TL::ND];

  __device__ __forceinline__ void scores(const unsigned char *kl, const unsigned char *vl, int n, f32x16 &p,
                                         f32x16 &dp, int lane) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = dp[i] = 0.f;
#pragma unroll
    for (int s = 0; s < TL::KS; ++s) mma_step<T>(TL::rows(kl, 32 * n, s, lane), qf[s], p);
#pragma unroll
    for (int s = 0; s < TL::KS; ++s) mma_step<T>(TL::rows(vl, 32 * n, s, lane), df[s], dp);
    if constexpr (sizeof(T) == 2) read_ahead<2 * TL::KS, 1, 1, 4>();
  }

  // delta = sum_j p (do . v_j) over the block's keys from `from` on (whole: over its tiles).
  __device__ __forceinline__ float delta_of_block(Lds &lds, int from, bool whole, int tid, int lane) const {
    const int h = lane >> 5;
    Stage<T, DH, BN, 256> sk, sv;
    float sum = 0.f;
    for (int kt = from; kt <= last; kt = whole ? win.after(kt) : kt + BN) {
      sk.fetch(kh, krow, kt, limit, hd, tid);
      sv.fetch(vh, vrow, kt, limit, hd, tid);
      sk.store(lds[0][0], tid);
      sv.store(lds[0][1], tid);
      __syncthreads();
#pragma unroll 1
      for (int n = 0; n < BN / 32; ++n) {
        f32x16 p, dp;
        scores(lds[0][0], lds[0][1], n, p, dp, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = kt + 32 * n + score_row(i, h);
          const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(p[i], c, -lse2)) * dp[i];
          if (win.sees(key)) sum += x;
        }
      }
      __syncthreads();
    }
    return half_sum(sum);
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int d = 0; d < TL::ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  }

  // A block of 32 keys, from kt on, at rows 32 n of the tiles.
  // (masked is no template argument: two copies of this body cost registers)
  template <bool GUARD>
  __device__ __forceinline__ void block(const unsigned char *kl, const unsigned char *vl, int n, int kt, bool masked,
                                        bool &met, int lane) {
    f32x16 p, dp;
    scores(kl, vl, n, p, dp, lane);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[i], c, -lse2)) * (dp[i] - delta);
    if (masked) {
      uint32_t seen = 0;
      win.masked(kt, qw, w_first, w_full, lane, [&](auto see) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool s = see(i);
          if (!s) p[i] = 0.f;
          seen |= (uint32_t)s << i;
        }
        if constexpr (WIN) asm volatile("" : "+v"(p));
      });
      if constexpr (GUARD || !STAGED) sum_rows_masked<GUARD, T, DH>(kl, 32 * n, p, seen, acc, met, lane);
    }
    if (!GUARD || !masked) {
      sum_rows<T, DH>(kl, 32 * n, p, acc, lane);
      if constexpr (sizeof(T) == 2) read_ahead<TL::PS * TL::ND, 2, 1, 4>();
    }
    if (REST && masked) sum_rows_rest<GUARD, T, DH>(kl, 32 * n, p, acc, lane);
  }

  // As delta_of_block, one tile of 32 keys from kt on (of a wave's share).
  __device__ __forceinline__ float delta_of_tile(unsigned char (&mine)[2][TL::bytes(32)], int kt, int lane) const {
    const int h = lane >> 5;
    Stage<T, DH, 32, 64> sk, sv;
    sk.fetch(kh, krow, kt, limit, hd, lane);
    sv.fetch(vh, vrow, kt, limit, hd, lane);
    sk.store(mine[0], lane);
    sv.store(mine[1], lane);
    wave_sync();
    f32x16 p, dp;
    scores(mine[0], mine[1], 0, p, dp, lane);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int key = kt + score_row(i, h);
      const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(p[i], c, -lse2)) * dp[i];
      if (win.sees(key)) sum += x;
    }
    wave_sync();
    return half_sum(sum);
  }

  // Every fourth tile of the block's keys, for one of its four waves; returns as pass().
  template <bool GUARD>
  __device__ __forceinline__ bool pass_few(unsigned char (&mine)[2][TL::bytes(32)], int wave, int lane) {
    static_assert(BN == 32, "");
    bool met = false;
    clear();
    Stage<T, DH, 32, 64> sk, sv;
    int t = wave, kt = win.tile(first, t);
    if (kt <= last) {
      sk.fetch(kh, krow, kt, limit, hd, lane);
      sv.fetch(vh, vrow, kt, limit, hd, lane);
      if constexpr (STAGED && !GUARD) met |= sk.not_finite();
      sk.store(mine[0], lane);
      sv.store(mine[1], lane);
    }
    for (; kt <= last;) {
      const int next = win.tile(first, t += 4);
      const bool more = next <= last;
      wave_sync();
      if (more) {
        sk.fetch(kh, krow, next, limit, hd, lane);
        sv.fetch(vh, vrow, next, limit, hd, lane);
      }
      block<GUARD>(mine[0], mine[1], 0, kt, REST || kt + 31 > qw || kt < w_full || win.part(kt, qw, w_first), met, lane);
      wave_sync();
      if (more) {
        if constexpr (STAGED && !GUARD) met |= sk.not_finite();
        sk.store(mine[0], lane);
        sv.store(mine[1], lane);
      }
      kt = next;
    }
    return met;
  }

  // All keys of the block; whether an infinity or a NaN in a masked tile was met (GUARD: never).
  template <bool GUARD>
  __device__ __forceinline__ bool pass(Lds &lds, int tid, int lane) {
    bool met = false;
    clear();
    Stage<T, DH, BN, 256> sk, sv;
    int buf = 0;
    if (first <= last) {
      sk.fetch(kh, krow, first, limit, hd, tid);
      sv.fetch(vh, vrow, first, limit, hd, tid);
      if constexpr (STAGED && !GUARD) met |= sk.not_finite();
      sk.store(lds[0][0], tid);
      sv.store(lds[0][1], tid);
    }
    __syncthreads();
    // the next tile comes in halves, so that only one of them is held in registers at a time
    for (int kt = first; kt <= last;) {
      const int next = win.after(kt);
      const bool more = next <= last;
      const bool work = kt <= qw + 31 && kt + BN > w_first && qw < limit && !win.none(kt, qw, w_first);
      const unsigned char *kl = lds[buf][0], *vl = lds[buf][1];
      const bool masked = kt + BN - 1 > qw || kt < w_full || win.part(kt, qw, w_first);
      if (more) sk.fetch(kh, krow, next, limit, hd, tid);
      if constexpr (GUARD || BN == 32) {
#pragma unroll 1
        for (int n = 0; n < BN / 32; ++n)
          if (work && !(n > 0 && win.half(kt))) block<GUARD>(kl, vl, n, kt + 32 * n, masked, met, lane);
        if (more) sv.fetch(vh, vrow, next, limit, hd, tid);
        if (STAGED && !GUARD && more) met |= sk.not_finite();
        if (more) sk.store(lds[buf ^ 1][0], tid);
      } else {
        if (work) block<GUARD>(kl, vl, 0, kt, masked, met, lane);
        if (more) {
          if constexpr (STAGED) met |= sk.not_finite();
          sk.store(lds[buf ^ 1][0], tid);
          sv.fetch(vh, vrow, next, limit, hd, tid);
        }
        if (work && !win.half(kt)) block<GUARD>(kl, vl, 1, kt + 32, masked, met, lane);
      }
      if (more) sv.store(lds[buf ^ 1][1], tid);
      __syncthreads();
      buf ^= 1;
      kt = next;
    }
    return met;
  }
};

// The block's and the wave's part of the problem: queries q0 .. q0 + rows - 1, the wave's
// from qw on; returns where the document of the block's last token starts.
template <typename T, int DH, int BN, bool REST, bool WIN>
__device__ __forceinline__ int begin(Dq<T, DH, BN, REST, WIN> &f, const AttnArgs &a, int bh, int q0, int rows, int qw, int lane) {
  using TL = Tile<T, DH>;
  const int b = bh / a.H, e = bh % a.H, g = e / (a.H / a.G), h = lane >> 5;
  f.kh = a.k.p + b * a.k.batch + g * a.k.head;
  f.vh = a.v.p + b * a.v.batch + g * a.v.head;
  f.krow = a.k.row;
  f.vrow = a.v.row;
  f.hd = a.hd;
  f.c = a.scale * kLog2e;
  f.qw = qw;
  f.limit = uniform(tokens_in_docs(a.cu, a.n_seqs, a.T));
  const int q = qw + (lane & 31);
  f.q = q;
  int tail, unused;
  doc_of(a.cu, a.n_seqs, a.T, f.limit, q, f.start, unused);
  keys_of(a.cu, a.n_seqs, a.T, f.limit, q0, rows, f.first, f.last);
  f.first = uniform(f.first);
  f.win.begin(a, q0, q, f.start, f.first);
  doc_of(a.cu, a.n_seqs, a.T, f.limit, f.last, tail, unused);
  f.w_first = uniform(f.start);  // (lane 0 has the lowest start)
  f.w_full = full_from(f.start, qw, f.limit);

  // a token of no document contributes nothing, whatever its rows hold
  const bool there = q < f.limit;
  const char *qrow = a.q.p + b * a.q.batch + e * a.q.head + (int64_t)q * a.q.row;
  const char *drow = a.d_o.p + b * a.d_o.batch + e * a.d_o.head + (int64_t)q * a.d_o.row;
  const char *orow = a.o.p + b * a.o.batch + e * a.o.head + (int64_t)q * a.o.row;
  f.delta = 0.f;
#pragma unroll
  for (int s = 0; s < TL::KS; ++s) {
    f.qf[s] = owned_chunk<T, DH>(qrow, there, 2 * s + h, a.hd);
    f.df[s] = owned_chunk<T, DH>(drow, there, 2 * s + h, a.hd);
    float x[TL::E], y[TL::E];
    widen<T>(f.df[s], x);
    widen<T>(owned_chunk<T, DH>(orow, there, 2 * s + h, a.hd), y);
#pragma unroll
    for (int i = 0; i < TL::E; ++i) f.delta = __builtin_fmaf(x[i], y[i], f.delta);
  }
  arrived(f.qf);
  arrived(f.df);
  f.delta = half_sum(f.delta);
  f.lse2 = INFINITY;  // log2 of the row's sum; +infinity: no key, every p is 0
  if (there) {
    const float v = a.lse[(int64_t)bh * a.T + q];
    if (v != -INFINITY) f.lse2 = v * kLog2e;
  }
  asm volatile("" : "+v"(f.lse2));
  return uniform(tail);
}

// Rows with few keys take delta = sum_j p (do . v_j) instead of do . o: o carries a rounding
// (2^-8 with bf16) that ds = p (do . v - delta) does not forgive where a few keys share the
// weight (two tokens of head_dim 16: dq 1.2 % off), while over many keys |o| falls below
// |v| and the error with it.  Done for rows whose document starts in the block or among the kBefore keys
// before it (so that no row of up to 64 keys takes the other, wherever its document lies in the
// row: 2 to 8 keys at the head of a block, heads of 64: dq 1.73 times as far off as its own rounding
// without them, 1.43 with them; 8192 tokens in 64 documents, 2 % of the training step); it costs blocks
// without such a start nothing.
// Through a window every row has few keys if the window and the sinks are no more than kBefore.
constexpr int kBefore = 64;
template <bool WIN>
__device__ __forceinline__ bool few_keys(const AttnArgs &a) {
  return WIN && (int64_t)a.window + a.sinks <= kBefore;
}
template <typename T, int DH, int BN, bool REST, bool WIN>
__global__ __launch_bounds__(256, (waves<T, DH>())) void attn_dq_kernel(AttnArgs a) {
  using F = Dq<T, DH, BN, REST, WIN>;
  __shared__ __align__(16) typename F::Lds lds;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = uniform(tid >> 6);
  int rank, bh;
  block_of(a.B * a.H, rank, bh);
  const int q0 = ((a.T + 127) / 128 - 1 - rank) * 128;
  F f;
  const int tail = begin(f, a, bh, q0, 128, q0 + wave * 32, lane);
  const bool whole = few_keys<WIN>(a);
  const int from = whole ? f.first : max(f.first, q0 - kBefore);
  if (f.first <= f.last && (whole || tail >= from)) {
    const float d = f.delta_of_block(lds, from, whole, tid, lane);
    if (whole || f.start >= from) f.delta = d;
  }
  if (f.q < a.T && h == 0) a.delta[(int64_t)bh * a.T + f.q] = f.delta;

  const bool met = f.template pass<false>(lds, tid, lane);
  if (__builtin_expect(__syncthreads_or(met), 0)) f.template pass<true>(lds, tid, lane);
  if (f.q >= f.limit) f.clear();
  if (f.q < a.T)
    write_row<T, DH>(a.dq.p + bh / a.H * a.dq.batch + bh % a.H * a.dq.head + (int64_t)f.q * a.dq.row, f.acc, a.scale,
                     a.hd, lane);
}

template <typename T, int DH, bool REST, bool WIN>
__global__ __launch_bounds__(256, sizeof(T) * DH > 256 ? 1 : 2) void attn_dq_few_kernel(AttnArgs a) {
  using F = Dq<T, DH, 32, REST, WIN>;
  __shared__ __align__(16) FewLds<T, DH> lds;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = uniform(tid >> 6);
  int rank, bh;
  block_of(a.B * a.H, rank, bh);
  const int q0 = ((a.T + 31) / 32 - 1 - rank) * 32;
  F f;
  const int tail = begin(f, a, bh, q0, 32, q0, lane);
  const bool whole = few_keys<WIN>(a);
  const int from = whole ? f.first : max(f.first, q0 - 96);
  if (f.first <= f.last && (whole || tail >= from)) {
    float d = 0.f;
    if constexpr (WIN) {
      // (tiles of one part up to 128 keys, of the sinks' and the window's part up to 160)
      for (int t = wave, kt; (kt = whole ? f.win.tile(from, t) : from + 32 * t) <= f.last; t += 4)
        d += f.delta_of_tile(lds.tile[wave], kt, lane);
    } else {
      const int kt = from + 32 * wave;
      d = kt <= f.last ? f.delta_of_tile(lds.tile[wave], kt, lane) : 0.f;
    }
    if (h == 0) lds.tot[wave][lane] = d;
    __syncthreads();
    if (whole || f.start >= from) {
      const int i = lane & 31;
      f.delta = (lds.tot[0][i] + lds.tot[1][i]) + (lds.tot[2][i] + lds.tot[3][i]);
    }
  }
  if (f.q < a.T && h == 0 && wave == 0) a.delta[(int64_t)bh * a.T + f.q] = f.delta;

  const bool met = f.template pass_few<false>(lds.tile[wave], wave, lane);
  if (__builtin_expect(__syncthreads_or(met), 0)) f.template pass_few<true>(lds.tile[wave], wave, lane);
  __syncthreads();  // (the sums take the tiles' place)
#pragma unroll
  for (int d = 0; d < F::TL::ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) lds.sum[wave][16 * d + i][lane] = f.acc[d][i];
  __syncthreads();
  if (f.q >= a.T) return;
  for (int d = wave; d < F::TL::ND; d += 4) {
    f32x16 x;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 16 * d + i;
      const float s = (lds.sum[0][r][lane] + lds.sum[1][r][lane]) + (lds.sum[2][r][lane] + lds.sum[3][r][lane]);
      x[i] = f.q < f.limit ? s : 0.f;
    }
    write_part<T>(a.dq.p + bh / a.H * a.dq.batch + bh % a.H * a.dq.head + (int64_t)f.q * a.dq.row, x, d, a.scale,
                  a.hd, lane);
  }
}

// The row of a sink in AttnArgs::far, [dk, dv][hd].
__device__ __forceinline__ float *far_row(const AttnArgs &a, int b, int g, int chunk, int start, int sink, int which) {
  const int64_t chunks = (a.T + a.far_chunk - 1) / a.far_chunk, n = far_slots(a);
  const int64_t slot = (((int64_t)b * a.G + g) * chunks + chunk) * n + (a.cu ? far_slot(a.far_chunk, chunk, start) : 0);
  return a.far + ((slot * a.sinks + sink) * 2 + which) * a.hd;
}
constexpr int kFarKeys = 32;  // sinks whose sums are joined at a time
template <int DH>
struct FarLds {
  float sum[kFarKeys][2][DH];
};

template <typename T, int DH, int BN, bool REST, bool WIN>
struct Dkv {
  using TL = Tile<T, DH>;
  static_assert(BN <= 64, "");
  struct Lds {
    unsigned char tile[2][2][TL::bytes(BN)];  // [buffer][query, do]
    float stat[2][2][BN];                    // lse log2 e (+infinity: no key) and delta of each query (FOLD: -lse / scale, -delta)
  };
  const AttnArgs &a;
  int b, e0, per;        // batch row, first query head, query heads
  int split;             // which part of the (head, query tile) pairs, of a.n_split
  int k0, stop, limit;   // the block: its first key, the last query + 1 that sees any, valid tokens
  int kw, w_end;         // the wave: its first key; up to w_end every key is seen
  int w_stop;            // no query from here on sees a key of the wave (WIN)
  int key, end;          // the lane's key and its document's end (WIN: the end of the queries that see it)
  float c;               // scale log2 e
  uint4 kf[TL::KS], vf[TL::KS];
  f32x16 ak[TL::ND], av[TL::ND];

  // With bf16 the sums of the scores start at -lse / scale and those of do . v at -delta, read from
  // LDS right into the accumulators, which saves their subtraction afterwards (fp32 sums
  // would lose a digit to it).
  static constexpr bool FOLD = sizeof(T) == 2;

  // What the sums of the scores and of do . v of the 32 queries at rows 32 n start from.
  __device__ __forceinline__ void begin(const float (&stat)[2][BN], int n, f32x16 &p, f32x16 &dp, int lane) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if constexpr (FOLD) {
        x = *reinterpret_cast<const float4 *>(&stat[0][32 * n + 8 * j + 4 * (lane >> 5)]);
        y = *reinterpret_cast<const float4 *>(&stat[1][32 * n + 8 * j + 4 * (lane >> 5)]);
      }
      p[4 * j] = x.x, p[4 * j + 1] = x.y, p[4 * j + 2] = x.z, p[4 * j + 3] = x.w;
      dp[4 * j] = y.x, dp[4 * j + 1] = y.y, dp[4 * j + 2] = y.z, dp[4 * j + 3] = y.w;
    }
  }
  // Probabilities in place of scores, ds in place of do . v, for four of them (register 4j on).
  __device__ __forceinline__ void weights(const float (&stat)[2][BN], int n, int j, f32x16 &p, f32x16 &dp,
                                          int lane) const {
    float4 l4 = make_float4(0.f, 0.f, 0.f, 0.f), d4 = l4;
    if constexpr (!FOLD) {
      l4 = *reinterpret_cast<const float4 *>(&stat[0][32 * n + 8 * j + 4 * (lane >> 5)]);
      d4 = *reinterpret_cast<const float4 *>(&stat[1][32 * n + 8 * j + 4 * (lane >> 5)]);
    }
    const float ls[4] = {l4.x, l4.y, l4.z, l4.w}, de[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = 4 * j + i;
      if constexpr (FOLD) {
        p[k] = __builtin_amdgcn_exp2f(p[k] * c);
        dp[k] *= p[k];
      } else {
        p[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[k], c, -ls[i]));
        dp[k] = p[k] * (dp[k] - de[i]);
      }
    }
  }
  // Which of the 32 queries from qt on see the lane's key; the others' scores to -infinity.
  __device__ __forceinline__ uint32_t hide(int qt, f32x16 &p, int lane) const {
    uint32_t seen = 0;
    const uint32_t reach = greater(0, end - key);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int q = qt + score_row(i, lane >> 5);
      const bool see = WIN ? (uint32_t)(q - key) < reach : q >= key && q < end;
      if (!see) p[i] = -INFINITY;
      seen |= (uint32_t)see << i;
    }
    return seen;
  }

  // Zeros for what is not seen (its p is 0 already, unless its query's lse is a NaN, but do . v may
  // have overflowed).
  static __device__ __forceinline__ void drop(uint32_t seen, f32x16 &p, f32x16 &dp) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(seen >> i & 1u)) p[i] = dp[i] = 0.f;
  }

  // The queries of one tile, from qt on.  Its products come in groups of three or four steps: scores and do . v
  // of the first 32 queries, those of the next 32, the sums of the first, the sums of the
  // next.  With one wave on a SIMD nobody else fills the gaps, so each group reads the operands of the
  // one after it before its products, and the softmax of 32 queries runs beside the products of a later
  // group; the scheduling barriers keep this order (left alone, every product waited for its own read).
  __device__ __forceinline__ void tile(const unsigned char *ql, const unsigned char *dl, const float (&stat)[2][BN],
                                       int qt, bool masked, bool &met, int lane) {
    constexpr int NB = BN / 32, S = TL::KS % 4 == 0 ? 4 : 3;         // blocks; steps of a group
    constexpr int GA = TL::KS / S, GC = TL::PS * TL::ND / S;          // groups of a score, of a sum
    static_assert(GA * S == TL::KS && GC * S == TL::PS * TL::ND, "");
    constexpr int C0 = NB * 2 * GA, ALL = C0 + NB * 2 * GC;
    f32x16 p[NB], dp[NB];
    uint32_t seen[NB];
    uint4 f[2][S];
    auto read = [&](int g, uint4(&x)[S]) {
      if (g < C0) {
        const unsigned char *t = g / GA % 2 == 0 ? ql : dl;
#pragma unroll
        for (int i = 0; i < S; ++i) x[i] = TL::rows(t, g / (2 * GA) * 32, g % GA * S + i, lane);
      } else {
        g -= C0;
        const unsigned char *t = g / GC % 2 == 0 ? dl : ql;
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int k = g % GC * S + i;
          x[i] = TL::cols(t, g / (2 * GC) * 32, k / TL::ND, k % TL::ND, lane);
        }
      }
    };
    auto multiply = [&](int g, const uint4(&x)[S]) {
      if (g < C0) {
        const int n = g / (2 * GA), s = g % GA * S;
#pragma unroll
        for (int i = 0; i < S; ++i) {
          if (g / GA % 2 == 0) mma_step<T>(x[i], kf[s + i], p[n]);
          else mma_step<T>(x[i], vf[s + i], dp[n]);
        }
      } else {
        g -= C0;
        const int n = g / (2 * GC);
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int k = g % GC * S + i;
          if (g / GC % 2 == 0) mma_step<T>(x[i], score_frag<T>(p[n], k / TL::ND), av[k % TL::ND]);
          else mma_step<T>(x[i], score_frag<T>(dp[n], k / TL::ND), ak[k % TL::ND]);
        }
      }
    };
    if (!WIN && masked) {
#pragma unroll
      for (int n = 0; n < NB; ++n) met |= not_finite<T, DH>(dl, 32 * n, lane) || not_finite<T, DH>(ql, 32 * n, lane);
    }
    read(0, f[0]);
#pragma unroll
    for (int n = 0; n < NB; ++n) begin(stat, n, p[n], dp[n], lane);
#pragma unroll
    for (int g = 0; g < ALL; ++g) {
      // scores just finished are masked, weights just finished cleared
      if (masked) {
        if (g % (2 * GA) == 0 && g > 0 && g <= C0) seen[g / (2 * GA) - 1] = hide(qt + g / (2 * GA) * 32 - 32, p[g / (2 * GA) - 1], lane);
        if (NB > 1 && g >= C0 && (g - C0) % (2 * GC) == 0) drop(seen[(g - C0) / (2 * GC)], p[(g - C0) / (2 * GC)], dp[(g - C0) / (2 * GC)]);
      }
      if (NB == 1 && g == C0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) weights(stat, 0, j, p[0], dp[0], lane);
        if (masked) drop(seen[0], p[0], dp[0]);
      }
      if (g + 1 < ALL) read(g + 1, f[(g + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
      multiply(g, f[g & 1]);
      if (NB > 1) {
        // the softmax of block n, spread over the groups from its scores to its sums
        const int from = g < C0 ? 2 * GA : C0, many = g < C0 ? 2 * GA : 2 * GC, n = g < C0 ? 0 : 1;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (g >= from && g < from + many && j * many / 4 == g - from) weights(stat, n, j, p[n], dp[n], lane);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (REST && masked) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        sum_rows_rest<false, T, DH>(dl, 32 * n, p[n], av, lane);
        sum_rows_rest<false, T, DH>(ql, 32 * n, dp[n], ak, lane);
      }
    }
  }
  // The same for 32 queries, sums guarded where some query does not see some key; or their rest.
  __device__ __forceinline__ void guarded(const unsigned char *ql, const unsigned char *dl,
                                          const float (&stat)[2][BN], int n, int qt, bool rest, int lane) {
    f32x16 p, dp;
    begin(stat, n, p, dp, lane);
#pragma unroll
    for (int s = 0; s < TL::KS; ++s) mma_step<T>(TL::rows(ql, 32 * n, s, lane), kf[s], p);
#pragma unroll
    for (int s = 0; s < TL::KS; ++s) mma_step<T>(TL::rows(dl, 32 * n, s, lane), vf[s], dp);
    const uint32_t seen = hide(qt, p, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) weights(stat, n, j, p, dp, lane);
    drop(seen, p, dp);
    if (REST && rest) {
      sum_rows_rest<true, T, DH>(dl, 32 * n, p, av, lane);
      sum_rows_rest<true, T, DH>(ql, 32 * n, dp, ak, lane);
    } else {
      sum_rows_guarded<T, DH>(dl, 32 * n, p, seen, av, lane);
      sum_rows_guarded<T, DH>(ql, 32 * n, dp, seen, ak, lane);
    }
  }

  // The block's part of the (head, query tile) pairs, heads outside; returns as Dq::pass.
  template <bool GUARD>
  __device__ __forceinline__ bool pass(Lds &lds, int tid, int lane) {
    bool met = false;
#pragma unroll
    for (int d = 0; d < TL::ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) ak[d][i] = av[d][i] = 0.f;
    Stage<T, DH, BN, 256> sq, sd;
    float st = 0.f;
    auto fetch = [&](int e, int qt) {
      sq.fetch(a.q.p + b * a.q.batch + e * a.q.head, a.q.row, qt, limit, a.hd, tid);
      sd.fetch(a.d_o.p + b * a.d_o.batch + e * a.d_o.head, a.d_o.row, qt, limit, a.hd, tid);
      if (tid < 2 * BN) {
        const int which = tid / BN, i = qt + tid % BN;
        const int64_t at = ((int64_t)b * a.H + e) * a.T + i;
        if (which == 0) {
          const float v = i < limit ? a.lse[at] : -INFINITY;
          st = v == -INFINITY ? INFINITY : FOLD ? v / a.scale : v * kLog2e;
        } else {
          st = i < limit ? a.delta[at] : 0.f;
        }
        if (FOLD) st = -st;
      }
    };
    auto store = [&](int to) {
      if constexpr (WIN && !GUARD) met |= sq.not_finite() || sd.not_finite();  // (as in the forward)
      sq.store(lds.tile[to][0], tid);
      sd.store(lds.tile[to][1], tid);
      if (tid < 2 * BN) lds.stat[to][tid / BN][tid % BN] = st;
    };
    const int n_q = k0 < stop ? (stop - k0 + BN - 1) / BN : 0;
    const int it0 = (int)((int64_t)n_q * per * split / a.n_split);
    const int it1 = (int)((int64_t)n_q * per * (split + 1) / a.n_split);
    int buf = 0, e = e0, qt = k0;
    if (it0 < it1) {
      e = e0 + it0 / n_q;
      qt = k0 + it0 % n_q * BN;
      fetch(e, qt);
      store(0);
    }
    __syncthreads();
    for (int it = it0; it < it1; ++it) {
      int e2 = e, qt2 = qt + BN;
      if (qt2 >= stop) {
        qt2 = k0;
        ++e2;
      }
      const bool more = it + 1 < it1;
      if (more) fetch(e2, qt2);
      if (qt + BN > kw && kw < limit && (!WIN || qt < w_stop)) {
        const unsigned char *ql = lds.tile[buf][0], *dl = lds.tile[buf][1];
        const bool masked = qt < kw + 31 || qt + BN > w_end;
        if constexpr (GUARD) {
#pragma unroll 1
          for (int i = 0; i < (REST && masked ? 2 : 1) * (BN / 32); ++i) {  // (sums in tile()'s order)
            const int n = i % (BN / 32);
            guarded(ql, dl, lds.stat[buf], n, qt + 32 * n, i >= BN / 32, lane);
          }
        } else {
          tile(ql, dl, lds.stat[buf], qt, masked, met, lane);
        }
      }
      if (more) store(buf ^ 1);
      __syncthreads();
      buf ^= 1;
      e = e2;
      qt = qt2;
    }
    return met;
  }

  // The chunks' sums of the sinks from s on, N values of a thread side by side, 8 or 16 loads on their way.
  template <int N>
  __device__ __forceinline__ void sum_far(FarLds<DH> &lds, int items, int c0, int c1, int g, int start, int s, int tid) {
    const int quads = a.hd / 4;
    for (int i0 = tid; i0 < items; i0 += 256 * N) {
      float4 sum[N];
      int kk[N], which[N], col[N];
#pragma unroll
      for (int m = 0; m < N; ++m) {
        const int i = lesser(i0 + 256 * m, items - 1);  // (past the end: the last one once more)
        kk[m] = i / (2 * quads);
        which[m] = i / quads % 2;
        col[m] = i % quads * 4;
        sum[m] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      constexpr int U = N == 1 ? 8 : 4;
      for (int c = c0; c < c1; c += U) {
        float4 x[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int m = 0; m < N; ++m)
            x[u][m] = *reinterpret_cast<const float4 *>(
                far_row(a, b, g, lesser(c + u, c1 - 1), start, s + kk[m] - start, which[m]) + col[m]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (c + u >= c1) break;
#pragma unroll
          for (int m = 0; m < N; ++m) {
            sum[m].x += x[u][m].x;
            sum[m].y += x[u][m].y;
            sum[m].z += x[u][m].z;
            sum[m].w += x[u][m].w;
          }
        }
      }
#pragma unroll
      for (int m = 0; m < N; ++m) *reinterpret_cast<float4 *>(&lds.sum[kk[m]][which[m]][col[m]]) = sum[m];
    }
  }

  // WIN: what attn_far_kernel has summed for the block's sinks, chunk by chunk, from the first query past the window's on
  // to doc_end, the end of their document.
  __device__ __forceinline__ void add_far(FarLds<DH> &lds, int g, int doc_end, int tid, int lane) {
    static_assert(sizeof(FarLds<DH>) <= sizeof(Lds), "");
    int start, unused;
    doc_of(a.cu, a.n_seqs, a.T, limit, lesser(k0 + 127, limit - 1), start, unused);
    start = uniform(start);
    const int s0 = greater(k0, start), s1 = lesser(k0 + 128, start + a.sinks);  // the block's sinks
    // (the splits of a block share the chunks)
    const int first = stop / a.far_chunk, chunks = (doc_end - 1) / a.far_chunk + 1 - first;
    const int c0 = first + chunks * split / a.n_split, c1 = first + chunks * (split + 1) / a.n_split;
    if (c0 == c1) return;
    const int quads = a.hd / 4;
    for (int s = s0; s < s1; s += kFarKeys) {
      const int n = lesser(kFarKeys, s1 - s);
      __syncthreads();
      const int items = n * 2 * quads;
      if (items <= 256) sum_far<1>(lds, items, c0, c1, g, start, s, tid);
      else sum_far<4>(lds, items, c0, c1, g, start, s, tid);
      __syncthreads();
      if (key >= s && key < s + n) {
#pragma unroll
        for (int d = 0; d < TL::ND; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int col = 32 * d + 8 * j + 4 * (lane >> 5);
            if (col >= a.hd) continue;
            const float4 x = *reinterpret_cast<const float4 *>(&lds.sum[key - s][0][col]);
            const float4 y = *reinterpret_cast<const float4 *>(&lds.sum[key - s][1][col]);
            ak[d][4 * j] += x.x, ak[d][4 * j + 1] += x.y, ak[d][4 * j + 2] += x.z, ak[d][4 * j + 3] += x.w;
            av[d][4 * j] += y.x, av[d][4 * j + 1] += y.y, av[d][4 * j + 2] += y.z, av[d][4 * j + 3] += y.w;
          }
      }
    }
  }
};

template <typename T, int DH, int BN, bool REST, bool WIN>
__global__ __launch_bounds__(256, DH == 64 && sizeof(T) == 2 ? 2 : 1) void attn_dkv_kernel(AttnArgs a) {
  using F = Dkv<T, DH, BN, REST, WIN>;
  using TL = Tile<T, DH>;
  __shared__ __align__(16) typename F::Lds lds;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = uniform(tid >> 6);
  const int group = a.H / a.G;  // query heads of a key/value head
  int rank, bg;
  block_of(a.B * a.G * a.n_split, rank, bg);
  const int b = bg / (a.G * a.n_split), gs = bg % (a.G * a.n_split), g = gs / a.n_split, split = gs % a.n_split;
  F f{a};
  f.b = b;
  f.per = group;
  f.e0 = g * group;
  f.split = split;
  f.k0 = rank * 128;
  f.c = a.scale * kLog2e;
  f.kw = f.k0 + wave * 32;
  f.limit = uniform(tokens_in_docs(a.cu, a.n_seqs, a.T));
  const int key = f.kw + (lane & 31);
  f.key = key;
  int start;
  doc_of(a.cu, a.n_seqs, a.T, f.limit, key, start, f.end);
  f.stop = uniform(queries_end(a.cu, a.n_seqs, a.T, f.limit, f.k0, 128));
  f.w_end = __builtin_amdgcn_readlane(f.end, 0);  // (the wave's ends rise)
  const int doc_end = f.stop;  // of the block's last key
  f.w_stop = 0;
  if constexpr (WIN) {
    // queries past the window's of the block see sinks alone, and come from attn_far_kernel
    f.stop = window_end(a.window, f.k0, 128, doc_end);
    if (key >= start + a.sinks) f.end = window_end(a.window, key, 1, f.end);
    f.end = lesser(f.end, f.stop);
    f.w_end = lesser(f.w_end, window_end(a.window, f.kw, 1, f.stop));
    int most = f.end;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) most = max(most, __shfl_xor(most, i));
    f.w_stop = uniform(most);
  }

  const bool there = key < f.limit;
  const char *krow = a.k.p + b * a.k.batch + g * a.k.head + (int64_t)key * a.k.row;
  const char *vrow = a.v.p + b * a.v.batch + g * a.v.head + (int64_t)key * a.v.row;
#pragma unroll
  for (int s = 0; s < TL::KS; ++s) {
    f.kf[s] = owned_chunk<T, DH>(krow, there, 2 * s + h, a.hd);
    f.vf[s] = owned_chunk<T, DH>(vrow, there, 2 * s + h, a.hd);
  }
  if constexpr (DH > 64) {
    arrived_acc(f.kf);
    arrived_acc(f.vf);
  } else {
    arrived(f.kf);
    arrived(f.vf);
  }
  const bool met = f.template pass<false>(lds, tid, lane);
  if (__builtin_expect(__syncthreads_or(met), 0)) f.template pass<true>(lds, tid, lane);
  if constexpr (WIN) {
    if (f.stop < doc_end && a.sinks > 0) f.add_far(*(FarLds<DH> *)&lds, g, doc_end, tid, lane);
  }
  if (key >= a.T) return;
  if (a.n_split == 1) {
    write_row<T, DH>(a.dk.p + b * a.dk.batch + g * a.dk.head + (int64_t)key * a.dk.row, f.ak, a.scale, a.hd, lane);
    write_row<T, DH>(a.dv.p + b * a.dv.batch + g * a.dv.head + (int64_t)key * a.dv.row, f.av, 1.f, a.hd, lane);
  } else {
    // [split][dk, dv][B][G][T][hd], fp32
    const int64_t rows = (int64_t)a.B * a.G * a.T, r = ((int64_t)b * a.G + g) * a.T + key;
    char *p0 = (char *)(a.part + ((int64_t)(2 * split) * rows + r) * a.hd);
    char *p1 = (char *)(a.part + ((int64_t)(2 * split + 1) * rows + r) * a.hd);
    write_row<float, DH>(p0, f.ak, a.scale, a.hd, lane);
    write_row<float, DH>(p1, f.av, 1.f, a.hd, lane);
  }
}

// dk and dv of sinks from the queries that see them past the window.  There are few such keys and up to a whole row
// of queries: a block takes the queries of a chunk for the query heads of one key/value head, its four waves
// every fourth tile of 32 of them against the same 32 keys, and joins their sums at the end.  Every tile's rows end
// with the queries that count, so what lies behind them is read as zeros.  Bound by latency and, with few sinks, by the
// tile of 32 that they are padded to (8192 tokens, 16 + 4 heads of 128: 19 us with 4 sinks, 46 with 128).
template <typename T, int DH>
struct FarTiles {
  unsigned char tile[4][2][Tile<T, DH>::bytes(32)];  // [wave][query, do]
  float stat[4][2][32];                              // lse log2 e (+infinity: no key) and delta
};
template <typename T, int DH, bool REST>
__global__ __launch_bounds__(256, 1) void attn_far_kernel(AttnArgs a) {
  using TL = Tile<T, DH>;
  __shared__ __align__(16) union {
    FarTiles<T, DH> in;
    float sum[4][DH / 2][64];  // [wave][accumulator register][lane]
  } lds;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = uniform(tid >> 6);
  const int chunks = (a.T + a.far_chunk - 1) / a.far_chunk;
  const int parts = far_parts(a), part = blockIdx.x / chunks % parts, bg = blockIdx.x / chunks / parts;
  const int chunk = blockIdx.x % chunks, g = bg % a.G, b = bg / a.G;
  const int limit = uniform(tokens_in_docs(a.cu, a.n_seqs, a.T));
  const int per = a.H / a.G;
  const float c = a.scale * kLog2e;
  for (int m = 0, done = -1; m < far_slots(a); ++m) {
    const int t = chunk * a.far_chunk + (m ? 128 * m - 1 : 0);
    int start, end;
    doc_of(a.cu, a.n_seqs, a.T, limit, t, start, end);
    start = uniform(start);
    end = uniform(end);
    if (end == 0 || start == done) continue;
    done = start;
    for (int s = start, n, group = 0; s < lesser(start + a.sinks, end); s += n, ++group) {
      const int k0 = s / 128 * 128;  // the block of attn_dkv_kernel that the sink is in
      n = lesser(lesser(start + a.sinks, k0 + 128) - s, 32);
      const int from = greater(chunk * a.far_chunk, window_end(a.window, k0, 128, end));
      const int to = lesser((chunk + 1) * a.far_chunk, end);
      if (from >= to || group % parts != part) continue;
      const int key = s + (lane & 31);
      const bool there = (lane & 31) < n;
      const char *krow = a.k.p + b * a.k.batch + g * a.k.head + (int64_t)key * a.k.row;
      const char *vrow = a.v.p + b * a.v.batch + g * a.v.head + (int64_t)key * a.v.row;
      uint4 kf[TL::KS], vf[TL::KS];
#pragma unroll
      for (int i = 0; i < TL::KS; ++i) {
        kf[i] = owned_chunk<T, DH>(krow, there, 2 * i + h, a.hd);
        vf[i] = owned_chunk<T, DH>(vrow, there, 2 * i + h, a.hd);
      }
      f32x16 ak[TL::ND], av[TL::ND];
      const int tiles = (to - from + 31) / 32, work = tiles * per;
      unsigned char(&ql)[TL::bytes(32)] = lds.in.tile[wave][0], (&dl)[TL::bytes(32)] = lds.in.tile[wave][1];
      float(&stat)[2][32] = lds.in.stat[wave];
      Stage<T, DH, 32, 64> sq, sd;
      float st = 0.f;
      auto fetch = [&](int it) {
        const int e = g * per + it / tiles, qt = from + it % tiles * 32;
        sq.fetch(a.q.p + b * a.q.batch + e * a.q.head, a.q.row, qt, to, a.hd, lane);
        sd.fetch(a.d_o.p + b * a.d_o.batch + e * a.d_o.head, a.d_o.row, qt, to, a.hd, lane);
        const int q = qt + (lane & 31);
        const int64_t at = ((int64_t)b * a.H + e) * a.T + q;
        if (h == 0) {
          const float v = q < to ? a.lse[at] : -INFINITY;
          st = v == -INFINITY ? INFINITY : v * kLog2e;
        } else {
          st = q < to ? a.delta[at] : 0.f;
        }
      };
      // The wave's tiles; whether it met an infinity or a NaN (REST; GUARD: never).  Every query sees every key here, so
      // these have their part in the first products: the others leave them out.
      auto pass = [&](auto guard) {
        constexpr bool GUARD = decltype(guard)::value;
        bool met = false;
#pragma unroll
        for (int d = 0; d < TL::ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) ak[d][i] = av[d][i] = 0.f;
        if (wave < work) fetch(wave);
        for (int it = wave; it < work; it += 4) {
          if constexpr (REST && !GUARD) met |= sq.not_finite() || sd.not_finite();
          wave_sync();
          sq.store(ql, lane);
          sd.store(dl, lane);
          stat[h][lane & 31] = st;
          wave_sync();
          if (it + 4 < work) fetch(it + 4);
          f32x16 p, dp;
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] = dp[i] = 0.f;
#pragma unroll
          for (int i = 0; i < TL::KS; ++i) mma_step<T>(TL::rows(ql, 0, i, lane), kf[i], p);
#pragma unroll
          for (int i = 0; i < TL::KS; ++i) mma_step<T>(TL::rows(dl, 0, i, lane), vf[i], dp);
          const int left = to - (from + it % tiles * 32);  // queries of the tile
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = score_row(i, h);
            p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[i], c, -stat[0][r]));
            dp[i] = p[i] * (dp[i] - stat[1][r]);
            if (r >= left) p[i] = dp[i] = 0.f;  // (a zero row times an infinite key is a NaN)
          }
#pragma unroll
          for (int x = 0; x < TL::PS; ++x) {
            const uint4 pf = score_frag<T>(p, x), df = score_frag<T>(dp, x);
#pragma unroll
            for (int d = 0; d < TL::ND; ++d) {
              mma_step<T>(TL::cols(dl, 0, x, d, lane), pf, av[d]);
              mma_step<T>(TL::cols(ql, 0, x, d, lane), df, ak[d]);
            }
          }
          if (REST) {
            sum_rows_rest<GUARD, T, DH>(dl, 0, p, av, lane);
            sum_rows_rest<GUARD, T, DH>(ql, 0, dp, ak, lane);
          }
        }
        return met;
      };
      const bool met = pass(std::false_type());
      if constexpr (REST) {
        if (__builtin_expect(__ballot(met) != 0, 0)) pass(std::true_type());
      }
      // the waves' sums, dk then dv
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int d = 0; d < TL::ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) lds.sum[wave][16 * d + i][lane] = which ? av[d][i] : ak[d][i];
        __syncthreads();
        if (there)
          for (int d = wave; d < TL::ND; d += 4) {
            f32x16 x;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int r = 16 * d + i;
              x[i] = (lds.sum[0][r][lane] + lds.sum[1][r][lane]) + (lds.sum[2][r][lane] + lds.sum[3][r][lane]);
            }
            write_part<float>((char *)far_row(a, b, g, chunk, start, key - start, which), x, d, 1.f, a.hd, lane);
          }
      }
      __syncthreads();
    }
  }
}

// dk and dv as the sums of their splits, in split order.
template <typename T>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int64_t rows = (int64_t)a.B * a.G * a.T;
  const int quads = a.hd / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= 2 * rows * quads) return;
  const int64_t which = i / (rows * quads), r = i / quads % rows;
  const int col = (int)(i % quads) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < a.n_split; ++k) {
    const float4 x = *reinterpret_cast<const float4 *>(a.part + ((2 * k + which) * rows + r) * a.hd + col);
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  const int64_t t = r % a.T, bg = r / a.T;
  const AttnView &v = which ? a.dv : a.dk;
  char *row = v.p + bg / a.G * v.batch + bg % a.G * v.head + t * v.row;
  if constexpr (sizeof(T) == 2) {
    bf16 w[4] = {(bf16)s.x, (bf16)s.y, (bf16)s.z, (bf16)s.w};
    *reinterpret_cast<uint2 *>(row + col * 2) = __builtin_bit_cast(uint2, *(const u32x2 *)w);
  } else {
    *reinterpret_cast<float4 *>(row + col * 4) = s;
  }
}

template <bool WIN, typename T, int DH, int BN, bool REST>
int launch_as(const AttnArgs &a, hipStream_t st) {
  const int n = (a.T + 127) / 128;
  if (few_blocks(a)) attn_dq_few_kernel<T, DH, REST, WIN><<<dim3((a.T + 31) / 32 * a.H * a.B), dim3(256), 0, st>>>(a);
  else attn_dq_kernel<T, DH, BN, REST, WIN><<<dim3(n * a.H * a.B), dim3(256), 0, st>>>(a);
  if constexpr (WIN) {
    if (has_far(a))
      attn_far_kernel<T, DH, REST><<<dim3((a.T + a.far_chunk - 1) / a.far_chunk * far_parts(a) * a.G * a.B), dim3(256), 0, st>>>(a);
  }
  attn_dkv_kernel<T, DH, BN, REST, WIN><<<dim3(n * a.G * a.n_split * a.B), dim3(256), 0, st>>>(a);
  if (a.n_split > 1) {
    const int64_t work = 2 * (int64_t)a.B * a.G * a.T * (a.hd / 4);
    attn_join_kernel<T><<<dim3((unsigned)((work + 255) / 256)), dim3(256), 0, st>>>(a);
  }
  return DYNCONV_OK;
}
template <bool WIN, typename T, int DH, int BN>
int launch(const AttnArgs &a, hipStream_t st) {
  const bool rest = WIN ? with_rest_window<T>(a) : with_rest<T>(a);
  return rest ? launch_as<WIN, T, DH, BN, sizeof(T) == 2>(a, st) : launch_as<WIN, T, DH, BN, false>(a, st);
}

// (Heads of 80 on 96 columns against 128, 16 + 4 heads, 4 rows of 4096 tokens: bf16 868 against 1010 us, fp32 6560
// against 8350.)
template <bool WIN>
int dispatch_bf16(const AttnArgs &a, hipStream_t st) {
  if (a.hd <= 64) return launch<WIN, bf16, 64, 64>(a, st);
  return a.hd <= 96 ? launch<WIN, bf16, 96, 64>(a, st) : launch<WIN, bf16, 128, 64>(a, st);
}
template <bool WIN>
int dispatch_fp32(const AttnArgs &a, hipStream_t st) {
  if (a.hd <= 32) return launch<WIN, float, 32, 64>(a, st);
  if (a.hd <= 64) return launch<WIN, float, 64, 32>(a, st);
  return a.hd <= 96 ? launch<WIN, float, 96, 32>(a, st) : launch<WIN, float, 128, 32>(a, st);
}

}  // namespace

}  // namespace dynconv
