// attn_paged_store.hip -- keys, turned, and values of whole prompts into the pages of a cache.
//
// Bound by memory: each element is read and written once.  A block takes a few tokens whole: while its
// threads' first vectors are on the way, others look up the tokens' pages and form the cosines and sines of each (token, pair)
// once, in LDS.  A token of no sequence, or whose page is not in the pool, is not written.  16384 tokens of 11 prompts, 4 heads
// of 128, bf16: 16.7 us, 4.0 TB/s; 37 tokens of 12 heads of 64: 4 us.
#include <algorithm>

#include "attn_paged.h"
#include "kernels.h"
#include "rope.h"

namespace dynconv {

namespace {

constexpr int kPairs = 1024, kTokens = 64;  // cosines and sines, and tokens, that a block holds

struct Place {
  int64_t k, v;  // bytes from the pools' starts, -1: the token is not stored
  int pos;
};

__device__ __forceinline__ Place place_of(const PagedStoreArgs &a, int64_t token) {
  Place p = {-1, -1, 0};
  int seq;
  const int pos = stored_at(a.cu, a.n_seqs, a.starts, a.counts, a.T, a.pages.capacity, token, seq);
  if (pos < 0) return p;
  const int page = page_at(a.pages.table + seq * a.pages.table_row, a.pages.size, a.pages.n_pages, pos);
  if (page < 0) return p;
  const int slot = pos % a.pages.size;
  p.k = page_row(a.pages.k, page, slot);
  p.v = page_row(a.pages.v, page, slot);
  p.pos = pos;
  return p;
}

template <int BYTES> struct Raw;
template <> struct Raw<16> { typedef uint4 type; };
template <> struct Raw<8> { typedef uint2 type; };
template <> struct Raw<4> { typedef uint32_t type; };
template <> struct Raw<2> { typedef uint16_t type; };

// Units of a head of k: rot / 2E of them turn two vectors of E elements, those after them copy two vectors each, and then those of v.
template <typename T, int E>
__global__ __launch_bounds__(256) void attn_paged_store_kernel(PagedStoreArgs a, int units_k, int units, int tokens) {
  typedef typename Raw<E * sizeof(T)>::type R;
  __shared__ float2 cs[kPairs];
  __shared__ Place places[kTokens];
  const int tid = threadIdx.x, pairs = a.rot / 2, turned = a.rot / (2 * E);
  const int64_t token0 = (int64_t)blockIdx.x * tokens, all = (int64_t)a.B * a.T;
  const int nt = (int)min((int64_t)tokens, all - token0), per = a.G * units, n = nt * per;
  for (int i0 = 0; i0 < n; i0 += 256) {
    const int i = i0 + tid;
    R x0, x1;
    int tok = 0, g = 0, u = 0, first = 0, second = 0;  // second: elements from the first vector to the other, 0: none
    if (i < n) {
      tok = i / per;
      g = (i - tok * per) / units;
      u = i - tok * per - g * units;
      const int64_t token = token0 + tok, b = token / a.T, t = token - b * a.T;
      if (u < turned) {
        first = a.interleaved ? 2 * u * E : u * E;
        second = a.interleaved ? E : pairs;
      } else {
        first = u < units_k ? a.rot + (u - turned) * 2 * E : (u - units_k) * 2 * E;
        second = first + E < a.hd ? E : 0;
      }
      const AttnView &w = u < units_k ? a.k : a.v;
      const char *x = w.p + b * w.batch + t * w.row + g * w.head + first * (int)sizeof(T);
      x0 = *(const R *)x;
      x1 = *(const R *)(x + second * (int)sizeof(T));
    }
    if (i0 == 0) {
      for (int j = tid; j < nt; j += 256) places[j] = place_of(a, token0 + j);
      __syncthreads();
      for (int j = tid; j < nt * pairs; j += 256) {
        float c, s;
        turn(places[j / pairs].pos, a.freqs[j % pairs], c, s);
        cs[j] = make_float2(c * a.factor, s * a.factor);
      }
      __syncthreads();
    }
    if (i >= n) continue;
    const Place &p = places[tok];
    if (p.k < 0) continue;
    if (u < turned) {
      const float2 *w = cs + tok * pairs + u * E;
      T xa[E], xb[E], ya[E], yb[E];
      __builtin_memcpy(xa, &x0, sizeof(R));
      __builtin_memcpy(xb, &x1, sizeof(R));
      float f, h;
      if (a.interleaved && E > 1) {
#pragma unroll
        for (int m = 0; m < E / 2; ++m) {
          turn_pair(to_f32(xa[2 * m]), to_f32(xa[2 * m + 1]), w[m].x, w[m].y, f, h);
          ya[2 * m] = from_f32<T>(f);
          ya[2 * m + 1] = from_f32<T>(h);
          turn_pair(to_f32(xb[2 * m]), to_f32(xb[2 * m + 1]), w[E / 2 + m].x, w[E / 2 + m].y, f, h);
          yb[2 * m] = from_f32<T>(f);
          yb[2 * m + 1] = from_f32<T>(h);
        }
      } else {
#pragma unroll
        for (int m = 0; m < E; ++m) {
          turn_pair(to_f32(xa[m]), to_f32(xb[m]), w[m].x, w[m].y, f, h);
          ya[m] = from_f32<T>(f);
          yb[m] = from_f32<T>(h);
        }
      }
      __builtin_memcpy(&x0, ya, sizeof(R));
      __builtin_memcpy(&x1, yb, sizeof(R));
    }
    char *y = (u < units_k ? a.pages.k.p + p.k + g * a.pages.k.head : a.pages.v.p + p.v + g * a.pages.v.head) + first * (int)sizeof(T);
    *(R *)y = x0;
    if (second) *(R *)(y + second * (int)sizeof(T)) = x1;
  }
}

constexpr int64_t kMaxBlocks = (1 << 24) - 1;  // of 256 threads, below 2^32 threads in all

template <typename T, int E>
int launch(const PagedStoreArgs &a, hipStream_t st) {
  const int units_k = a.rot / (2 * E) + ((a.hd - a.rot) / E + 1) / 2, units = units_k + (a.hd / E + 1) / 2;
  // two units for a thread, no more tokens than leave a block for every CU or fit the block's tables
  const int64_t all = (int64_t)a.B * a.T;
  const int64_t tokens = std::max<int64_t>(1, std::min<int64_t>({(512 + a.G * units - 1) / (a.G * units), all / 256, kTokens,
                                                                 a.rot ? kPairs / (a.rot / 2) : kTokens}));
  const int64_t blocks = (all + tokens - 1) / tokens;
  if (blocks > kMaxBlocks) return DYNCONV_E_LIMIT;
  attn_paged_store_kernel<T, E><<<dim3((unsigned)blocks), dim3(256), 0, st>>>(a, units_k, units, (int)tokens);
  return DYNCONV_OK;
}

}  // namespace

int attn_paged_store(const PagedStoreArgs &a, int dtype, int vec_bytes, hipStream_t st) {
  if (dtype == DYNCONV_BF16) {
    if (vec_bytes == 16) return launch<bf16, 8>(a, st);
    return vec_bytes == 8 ? launch<bf16, 4>(a, st) : launch<bf16, 1>(a, st);
  }
  if (vec_bytes == 16) return launch<float, 4>(a, st);
  return vec_bytes == 8 ? launch<float, 2>(a, st) : launch<float, 1>(a, st);
}

}  // namespace dynconv
