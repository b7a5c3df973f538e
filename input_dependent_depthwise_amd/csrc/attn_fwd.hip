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
constexpr float kSlack = 8.f;

template <typename T, int DH, int BN>
__global__ __launch_bounds__(256, 2) void attn_fwd_kernel(AttnArgs a) {
  using TL = Tile<T, DH>;
  __shared__ __align__(16) unsigned char lds[2][2][BN * TL::ROW];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = uniform(tid >> 6);
  int rank, bh;
  block_of(a.B * a.H, rank, bh);
  const int n_tiles = (a.T + 127) / 128;
  const int q0 = (n_tiles - 1 - rank) * 128;
  const int b = bh / a.H, e = bh % a.H, g = e / (a.H / a.G);
  const char *kh = a.k.p + b * a.k.batch + g * a.k.head;
  const char *vh = a.v.p + b * a.v.batch + g * a.v.head;

  const int qw = q0 + wave * 32, q = qw + (lane & 31);
  const int limit = uniform(tokens_in_docs(a.cu, a.n_seqs, a.T));
  int start, end;
  doc_of(a.cu, a.n_seqs, a.T, q, start, end);
  int first, unused;
  doc_of(a.cu, a.n_seqs, a.T, q0, first, unused);
  first = uniform(first);
  const int last = min(q0 + 127, limit - 1);             // the block's last key
  const int w_first = uniform(start);                    // the wave's first key (its lane 0 has the lowest start)
  const int w_full = __builtin_amdgcn_readlane(start, 31);  // from here on every row of the wave sees keys

  uint4 qf[TL::KS];
  const char *qrow = a.q.p + b * a.q.batch + e * a.q.head + (int64_t)q * a.q.row;
#pragma unroll
  for (int s = 0; s < TL::KS; ++s) qf[s] = owned_chunk<T, DH>(qrow, q < a.T, 2 * s + h, a.hd);

  f32x16 acc[TL::ND];
#pragma unroll
  for (int d = 0; d < TL::ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;
  const float c = a.scale * kLog2e;

  Stage<T, DH, BN, 256> sk, sv;
  int buf = 0;
  if (first <= last) {
    sk.fetch(kh, a.k.row, first, limit, a.hd, tid);
    sv.fetch(vh, a.v.row, first, limit, a.hd, tid);
    sk.store(lds[0][0], tid);
    sv.store(lds[0][1], tid);
  }
  __syncthreads();
  for (int kt = first; kt <= last; kt += BN) {
    const bool more = kt + BN <= last;
    if (more) {
      sk.fetch(kh, a.k.row, kt + BN, limit, a.hd, tid);
      sv.fetch(vh, a.v.row, kt + BN, limit, a.hd, tid);
    }
    if (kt <= qw + 31 && kt + BN > w_first && qw < limit) {
      const unsigned char *kl = lds[buf][0], *vl = lds[buf][1];
      f32x16 p[BN / 32];
#pragma unroll
      for (int n = 0; n < BN / 32; ++n) {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[n][i] = 0.f;
#pragma unroll
        for (int s = 0; s < TL::KS; ++s) mma_step<T>(TL::rows(kl, 32 * n, s, lane), qf[s], p[n]);
      }
      const bool masked = kt + BN - 1 > qw || kt < w_full;
      uint32_t seen[BN / 32];
#pragma unroll
      for (int n = 0; n < BN / 32; ++n) seen[n] = 0xffff;
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
#pragma unroll
      for (int n = 0; n < BN / 32; ++n) sum_rows<T, DH>(vl, 32 * n, p[n], masked, seen[n], acc, lane);
    }
    if (more) {
      sk.store(lds[buf ^ 1][0], tid);
      sv.store(lds[buf ^ 1][1], tid);
    }
    __syncthreads();
    buf ^= 1;
  }
  l = half_sum(l);
  if (q < a.T) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    write_row<T, DH>(a.o.p + b * a.o.batch + e * a.o.head + (int64_t)q * a.o.row, acc, inv, a.hd, lane);
    if (a.lse && h == 0)
      a.lse[(int64_t)bh * a.T + q] = l == 0.f ? -INFINITY : m * a.scale + __builtin_amdgcn_logf(l) * kLn2;
  }
}

template <typename T, int DH, int BN>
int launch(const AttnArgs &a, hipStream_t st) {
  const int n = (a.T + 127) / 128 * a.H * a.B;
  attn_fwd_kernel<T, DH, BN><<<dim3(n), dim3(256), 0, st>>>(a);
  return DYNCONV_OK;
}

}  // namespace

int attn_fwd(const AttnArgs &a, int dtype, hipStream_t st) {
  if (dtype == DYNCONV_BF16) return a.hd <= 64 ? launch<bf16, 64, 64>(a, st) : launch<bf16, 128, 64>(a, st);
  return a.hd <= 64 ? launch<float, 64, 32>(a, st) : launch<float, 128, 32>(a, st);
}

}  // namespace dynconv
