// attn_fwd.hip -- causal attention over whole sequences, forward.
//
// o[i] = sum_j exp(s[i,j] - lse[i]) v[j],  s = scale q[i].k[j],  j <= i in i's
// document, in one pass over the keys with a running maximum and sum.
#include "attn.h"
#include "kernels.h"

namespace dynconv {

namespace {

// A block has 4 waves of 32 queries of one head; key and value tiles of BN rows
// are double-buffered in LDS (one barrier a tile; the loads of the next tile
// fly while this one is computed).  The running maximum is raised only when a
// score passes it by 2^kSlack (a sum of exp2(<= 8) keeps its relative error),
// so the accumulator is rarely rescaled.
//
// Bound by the matrix and the vector units, which two waves of a SIMD use in turn: 16 + 4 heads of
// 128, 4 rows of 4096 tokens, bf16: 304 us, 0.90 PFLOP/s (47 % of the matrix cores' cycles, 45 % of the
// vector units'); 12 heads of 64, 8 rows of 2048: 75 to 78 us with the card, 0.67 PFLOP/s, the vector units 66 %
// busy with the exponentials and what surrounds them.  Tiles of 64 keys: 32 took 96 us where 64
// take 82 (heads of 64, two waves), 128 took 123 (registers).
constexpr float kSlack = 8.f;

template <typename T, int DH, int BN, bool REST>
struct Fwd {
  using TL = Tile<T, DH>;
  typedef unsigned char Lds[2][2][TL::bytes(BN)];  // [buffer][key, value]
  // the block: keys of its head, their range, valid tokens
  const char *kh, *vh;
  int64_t krow, vrow;
  int first, last, limit, hd;
  // the wave: its first query, first key, and the key from which on every row sees keys
  int qw, w_first, w_full;
  int q, start;  // the lane's query and its document's start
  float c;       // scale log2 e
  uint4 qf[TL::KS];
  f32x16 acc[TL::ND];
  float m, l;

  static __device__ __forceinline__ uint4 chunk(const char *row, bool there, int chunk, int hd) {
    return owned_chunk<T, DH>(row, there, chunk, hd);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int d = 0; d < TL::ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  }

  // The keys of one tile, from kt on.
  template <bool GUARD>
  __device__ __forceinline__ void step(const unsigned char *kl, const unsigned char *vl, int kt, bool &met, int lane) {
    const int h = lane >> 5;
    const bool masked = (REST && BN == 32) || kt + BN - 1 > qw || kt < w_full;
    f32x16 p[BN / 32];
#pragma unroll
    for (int n = 0; n < BN / 32; ++n) {
#pragma unroll
      for (int i = 0; i < 16; ++i) p[n][i] = 0.f;
#pragma unroll
      for (int s = 0; s < TL::KS; ++s) mma_step<T>(TL::rows(kl, 32 * n, s, lane), qf[s], p[n]);
    }
    if constexpr (sizeof(T) == 2) read_ahead<BN / 32 * TL::KS, 1, 1, 4>();
    uint32_t seen[BN / 32];
    if (masked) {
#pragma unroll
      for (int n = 0; n < BN / 32; ++n) {
        seen[n] = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = kt + 32 * n + score_row(i, h);
          const bool see = key <= q && key >= start;
          if (!see) p[n][i] = -INFINITY;
          seen[n] |= (uint32_t)see << i;
        }
      }
    }
    float mx = p[0][0];
#pragma unroll
    for (int n = 0; n < BN / 32; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, p[n][i]);
    mx = half_max(mx);
    const bool raise = mx > m && !((mx - m) * c <= kSlack);  // (by row: no row's sums depend on another's)
    if (__ballot(raise) != 0) {
      const float up = raise ? mx : m;
      const float f = raise ? __builtin_amdgcn_exp2f((m - up) * c) : 1.f;
      m = up;
      l *= f;
#pragma unroll
      for (int d = 0; d < TL::ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] *= f;
    }
    const float mc = m == -INFINITY ? 0.f : m * c;
#pragma unroll
    for (int n = 0; n < BN / 32; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[n][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[n][i], c, -mc));
        l += p[n][i];
      }
    if (masked) {
#pragma unroll
      for (int n = 0; n < BN / 32; ++n)
        sum_rows_masked<GUARD, T, DH>(vl, 32 * n, p[n], seen[n], acc, met, lane);
    }
    if (!GUARD || !masked) {
#pragma unroll
      for (int n = 0; n < BN / 32; ++n) {
        sum_rows<T, DH>(vl, 32 * n, p[n], acc, lane);
        if constexpr (sizeof(T) == 2) read_ahead<TL::PS * TL::ND, 2, 1, 4>();
      }
    }
    if (REST && masked) {
#pragma unroll
      for (int n = 0; n < BN / 32; ++n) sum_rows_rest<GUARD, T, DH>(vl, 32 * n, p[n], acc, lane);
    }
  }

  // Every fourth tile of the block's keys, for one of its four waves; returns as pass().
  template <bool GUARD>
  __device__ __forceinline__ bool pass_few(unsigned char (&mine)[2][TL::bytes(32)], int wave, int lane) {
    static_assert(BN == 32, "");
    bool met = false;
    m = -INFINITY;
    l = 0.f;
    clear();
    Stage<T, DH, 32, 64> sk, sv;
    int kt = first + 32 * wave;
    if (kt <= last) {
      sk.fetch(kh, krow, kt, limit, hd, lane);
      sv.fetch(vh, vrow, kt, limit, hd, lane);
      sk.store(mine[0], lane);
      sv.store(mine[1], lane);
    }
    for (; kt <= last; kt += 128) {
      const bool more = kt + 128 <= last;
      wave_sync();
      if (more) {
        sk.fetch(kh, krow, kt + 128, limit, hd, lane);
        sv.fetch(vh, vrow, kt + 128, limit, hd, lane);
      }
      step<GUARD>(mine[0], mine[1], kt, met, lane);
      wave_sync();
      if (more) {
        sk.store(mine[0], lane);
        sv.store(mine[1], lane);
      }
    }
    return met;
  }

  // All keys of the block; whether an infinity or a NaN in a masked tile was met (GUARD: never).
  template <bool GUARD>
  __device__ __forceinline__ bool pass(Lds &lds, int tid, int lane) {
    bool met = false;
    m = -INFINITY;
    l = 0.f;
    clear();
    Stage<T, DH, BN, 256> sk, sv;
    int buf = 0;
    if (first <= last) {
      sk.fetch(kh, krow, first, limit, hd, tid);
      sv.fetch(vh, vrow, first, limit, hd, tid);
      sk.store(lds[0][0], tid);
      sv.store(lds[0][1], tid);
    }
    __syncthreads();
    for (int kt = first; kt <= last; kt += BN) {
      const bool more = kt + BN <= last;
      if (more) {
        sk.fetch(kh, krow, kt + BN, limit, hd, tid);
        sv.fetch(vh, vrow, kt + BN, limit, hd, tid);
      }
      if (kt <= qw + 31 && kt + BN > w_first && qw < limit) {
        const unsigned char *kl = lds[buf][0], *vl = lds[buf][1];
        step<GUARD>(kl, vl, kt, met, lane);
      }
      if (more) {
        sk.store(lds[buf ^ 1][0], tid);
        sv.store(lds[buf ^ 1][1], tid);
      }
      __syncthreads();
      buf ^= 1;
    }
    return met;
  }
};

// The block's and the wave's part of the problem: queries q0 .. q0 + rows - 1, the wave's from qw on.
template <typename F>
__device__ __forceinline__ void begin(F &f, const AttnArgs &a, int bh, int q0, int rows, int qw, int lane) {
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
  int unused;
  doc_of(a.cu, a.n_seqs, a.T, f.limit, q, f.start, unused);
  keys_of(a.cu, a.n_seqs, a.T, f.limit, q0, rows, f.first, f.last);
  f.first = uniform(f.first);
  f.w_first = uniform(f.start);  // (lane 0 has the lowest start)
  f.w_full = full_from(f.start, qw, f.limit);
  const char *qrow = a.q.p + b * a.q.batch + e * a.q.head + (int64_t)q * a.q.row;
#pragma unroll
  for (int s = 0; s < F::TL::KS; ++s) f.qf[s] = F::chunk(qrow, q < a.T, 2 * s + h, a.hd);
  arrived(f.qf);
}

template <typename T, int DH, int BN, bool REST>
__global__ __launch_bounds__(256, (waves<T, DH>())) void attn_fwd_kernel(AttnArgs a) {
  using F = Fwd<T, DH, BN, REST>;
  __shared__ __align__(16) typename F::Lds lds;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = uniform(tid >> 6);
  int rank, bh;
  block_of(a.B * a.H, rank, bh);
  const int q0 = ((a.T + 127) / 128 - 1 - rank) * 128;
  F f;
  begin(f, a, bh, q0, 128, q0 + wave * 32, lane);
  const bool met = f.template pass<false>(lds, tid, lane);
  if (__builtin_expect(__syncthreads_or(met), 0)) f.template pass<true>(lds, tid, lane);

  const float l = half_sum(f.l);
  if (f.q < a.T) {
    const bool none = f.q >= f.limit || l == 0.f;  // no keys
    if (none) f.clear();
    const float inv = none ? 0.f : 1.f / l;
    write_row<T, DH>(a.o.p + bh / a.H * a.o.batch + bh % a.H * a.o.head + (int64_t)f.q * a.o.row, f.acc, inv, a.hd, lane);
    if (a.lse && h == 0)
      a.lse[(int64_t)bh * a.T + f.q] = none ? -INFINITY : f.m * a.scale + __builtin_amdgcn_logf(l) * kLn2;
  }
}

template <typename T, int DH, bool REST>
__global__ __launch_bounds__(256, sizeof(T) * DH > 256 ? 1 : 2) void attn_fwd_few_kernel(AttnArgs a) {
  using F = Fwd<T, DH, 32, REST>;
  __shared__ __align__(16) FewLds<T, DH> lds;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = uniform(tid >> 6);
  int rank, bh;
  block_of(a.B * a.H, rank, bh);
  const int q0 = ((a.T + 31) / 32 - 1 - rank) * 32;
  F f;
  begin(f, a, bh, q0, 32, q0, lane);
  const bool met = f.template pass_few<false>(lds.tile[wave], wave, lane);
  if (__builtin_expect(__syncthreads_or(met), 0)) f.template pass_few<true>(lds.tile[wave], wave, lane);
  __syncthreads();  // (the sums take the tiles' place)
  const float own = half_sum(f.l);
  if (h == 0) {
    lds.top[wave][lane] = f.m;
    lds.tot[wave][lane] = own;
  }
#pragma unroll
  for (int d = 0; d < F::TL::ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) lds.sum[wave][16 * d + i][lane] = f.acc[d][i];
  __syncthreads();
  if (f.q >= a.T) return;
  float part[4], top = -INFINITY, l = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, lds.top[w][lane & 31]);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float m = lds.top[w][lane & 31], t = lds.tot[w][lane & 31];
    part[w] = m == -INFINITY ? (t == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f((m - top) * f.c);
    l = __builtin_fmaf(part[w], t, l);
  }
  const bool none = f.q >= f.limit || l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  for (int d = wave; d < F::TL::ND; d += 4) {
    f32x16 x;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) s = __builtin_fmaf(part[w], lds.sum[w][16 * d + i][lane], s);
      x[i] = none ? 0.f : s;
    }
    write_part<T>(a.o.p + bh / a.H * a.o.batch + bh % a.H * a.o.head + (int64_t)f.q * a.o.row, x, d, inv, a.hd, lane);
  }
  if (a.lse && wave == 0 && h == 0)
    a.lse[(int64_t)bh * a.T + f.q] = none ? -INFINITY : top * a.scale + __builtin_amdgcn_logf(l) * kLn2;
}

template <typename T, int DH, int BN, bool REST>
int launch_as(const AttnArgs &a, hipStream_t st) {
  if (few_blocks(a)) {
    attn_fwd_few_kernel<T, DH, REST><<<dim3((a.T + 31) / 32 * a.H * a.B), dim3(256), 0, st>>>(a);
    return DYNCONV_OK;
  }
  attn_fwd_kernel<T, DH, BN, REST><<<dim3((a.T + 127) / 128 * a.H * a.B), dim3(256), 0, st>>>(a);
  return DYNCONV_OK;
}
template <typename T, int DH, int BN>
int launch(const AttnArgs &a, hipStream_t st) {
  return with_rest<T>(a) ? launch_as<T, DH, BN, sizeof(T) == 2>(a, st) : launch_as<T, DH, BN, false>(a, st);
}

}  // namespace

// Tiles of the least width that holds the head, the columns past it zeros: heads of 80 on 96 columns
// against 128 (16 + 4 heads, 4 rows of 4096 tokens) bf16 240 against 266 us, fp32 2020 against 2510.
int attn_fwd(const AttnArgs &a, int dtype, hipStream_t st) {
  if (dtype == DYNCONV_BF16) {
    if (a.hd <= 64) return launch<bf16, 64, 64>(a, st);
    return a.hd <= 96 ? launch<bf16, 96, 64>(a, st) : launch<bf16, 128, 64>(a, st);
  }
  if (a.hd <= 32) return launch<float, 32, 64>(a, st);
  if (a.hd <= 64) return launch<float, 64, 32>(a, st);
  return a.hd <= 96 ? launch<float, 96, 32>(a, st) : launch<float, 128, 32>(a, st);
}

}  // namespace dynconv
