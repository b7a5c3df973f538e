// attn_paged.hip -- attention of one new token per sequence over a cache kept in pages.
//
// Bound by the cache: every key and value row that is seen is read once.  A unit of work is a sequence and a
// key/value head with up to 16 of its query heads; its groups are the new token (group 0), then 32 cached tokens each:
// those that hold sinks before the window, and those from the window's first one on.  A wave takes a group
// straight from memory to registers (attn_group.h); lane l looks up the page of key l and forms the addresses
// of its key and value, and the lanes that load the row get them from it, so pages of any size
// may start and end anywhere in a group.  A key that is not seen, or whose page is not in the pool, has the address of a
// row of zeros and a score of -infinity.  The table's entries of the group after next are on their way while
// the next group's rows are.
//
// Lengths differ, and the host does not know them.  Flattened launch: the units' groups stand in one row, each block
// finds its equal share of them from the lengths (a sum over the batch in LDS) and takes the units that lie in it one after
// another.  A unit that several blocks share is joined by a second kernel, in the order of the blocks.
#include <algorithm>
#include <type_traits>

#include "attn_group.h"
#include "attn_paged.h"
#include "kernels.h"
#include "rope.h"

namespace dynconv {

namespace {

constexpr int kMostSeqs = 1024;  // whose lengths a block of the flattened launch adds up

__device__ const uint4 kZeroRow[32] = {};  // stands for a row that is not there

// The page of the lane's key (lane & 31) in a group, -1 where the key is not seen.
__device__ __forceinline__ int page_of(const PagedArgs &a, const int32_t *table, const Seen &s, int group, int lane) {
  const int key = first_key(s, group) + (lane & 31);
  return sees(s, key) ? table[(uint32_t)key / (uint32_t)a.pages.size] : -1;
}

typedef const u32x4 __attribute__((address_space(1))) *Global16;
typedef const u32x2 __attribute__((address_space(1))) *Global8;

__device__ __forceinline__ const char *from_lane(const char *p, int lane) {
  return (const char *)__shfl((unsigned long long)p, lane);
}

// The group's rows from their lanes' pages; returns which keys there are (uniform).
template <typename T, int DH>
__device__ __forceinline__ uint32_t fetch(Group<T, DH> &x, const PagedArgs &a, const Seen &s, int g, int group, int page,
                                          int lane) {
  using G = Group<T, DH>;
  const int m = lane & 15, u = lane >> 4;
  const bool there = (uint32_t)page < (uint32_t)a.pages.n_pages;
  const uint32_t mask = (uint32_t)__ballot(there);
  const char *zero = (const char *)kZeroRow;
  const int slot = (int)((uint32_t)(first_key(s, group) + (lane & 31)) % (uint32_t)a.pages.size);
  const char *kr = there ? a.pages.k.p + page_row(a.pages.k, page, slot) + g * a.pages.k.head : zero;
  const char *vr = there ? a.pages.v.p + page_row(a.pages.v, page, slot) + g * a.pages.v.head : zero;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const char *row = from_lane(kr, 8 * (m >> 2) + 4 * t + (m & 3));
#pragma unroll
    for (int i = 0; i < G::NS; ++i) {
      const int chunk = 4 * i + u;
      const u32x4 w = *(Global16)(chunk * G::E < a.hd ? row + chunk * 16 : zero);
      x.k[t][i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const char *row = from_lane(vr, 8 * u + i);
    if constexpr (G::VW == 2) {
      const u32x2 w = *(Global8)(m * G::EV < a.hd ? row + m * G::EV * (int)sizeof(T) : zero);
      x.v[i][0] = w[0];
      x.v[i][1] = w[1];
    } else {
#pragma unroll
      for (int j = 0; j < G::VW / 4; ++j) {
        const u32x4 w = *(Global16)(m * G::EV + j * G::E < a.hd ? row + m * G::EV * (int)sizeof(T) + 16 * j : zero);
#pragma unroll
        for (int c = 0; c < 4; ++c) x.v[i][4 * j + c] = w[c];
      }
    }
  }
  return mask;
}

template <typename T, int DH, int WAVES>
struct Step {
  static constexpr int THREADS = WAVES * 64, LD = DH + 4;  // (rows shifted by 16 bytes against bank conflicts)
  using GP = Group<T, DH>;
  struct Lds {
    float q[17][LD];  // 16 query heads times scale log2 e, then the new key
    float tops[WAVES][16], tots[WAVES][16];
    float sums[1];  // [wave][column][LD]
  };
  static size_t lds_bytes(int cols) { return sizeof(Lds) + (size_t)WAVES * cols * LD * 4; }

  // Groups s0 .. s1 - 1 of a unit (sequence b with n cached tokens, key/value head g, column block cb); the result as o, or as
  // sums and statistics at `slot`.
  static __device__ __forceinline__ void run(const PagedArgs &a, Lds &lds, int b, const Seen &seen, int g, int cb, int s0,
                                             int s1, int slot, int tid) {
    const int lane = tid & 63, wave = uniform(tid >> 6);
    const int per = a.H / a.G, n = seen.n;
    const int e0 = g * per + cb * 16, cols = min(16, per - cb * 16);
    const int32_t *table = a.pages.table + b * a.pages.table_row;
    const int first = s0 + wave == 0 ? WAVES : s0 + wave;  // (the new token is no group of the cache)
    GP x;
    uint32_t mask = 0;
    int page = -1;
    if (first < s1) {
      mask = fetch(x, a, seen, g, first, page_of(a, table, seen, first, lane), lane);
      if (first + WAVES < s1) page = page_of(a, table, seen, first + WAVES, lane);
    }
    __syncthreads();  // (the unit before this one has been written)
    for (int i = tid; i < 17 * LD; i += THREADS) (&lds.q[0][0])[i] = 0.f;
    __syncthreads();
    // q and the new key, turned, in LDS; the new key and value into their page
    const float c = a.scale * kLog2e;
    const int half = a.hd / 2;
    const int at = s0 == 0 && cb == 0 ? page_at(table, a.pages.size, a.pages.n_pages, n) : -1;
    for (int i = tid; i < (cols + 1) * half; i += THREADS) {
      const int hh = i / half, p = i % half;
      const bool key = hh == cols;
      const T *src = key ? (const T *)(a.k.p + b * a.k.batch + g * a.k.head)
                         : (const T *)(a.q.p + b * a.q.batch + (e0 + hh) * a.q.head);
      int i0 = 2 * p, i1 = 2 * p + 1;  // (rot is even: the rest starts at 2 (rot/2))
      float cs = 1.f, sn = 0.f;
      if (p < a.rot / 2) {
        i0 = a.interleaved ? 2 * p : p;
        i1 = a.interleaved ? 2 * p + 1 : p + a.rot / 2;
        turn(n, a.freqs[p], cs, sn);
        cs *= a.factor;
        sn *= a.factor;
      }
      const float u = to_f32(src[i0]), w = to_f32(src[i1]);
      float r0 = u, r1 = w;
      if (p < a.rot / 2) turn_pair(u, w, cs, sn, r0, r1);
      if (key) {
        const T k0 = from_f32<T>(r0), k1 = from_f32<T>(r1);
        lds.q[16][i0] = to_f32(k0);
        lds.q[16][i1] = to_f32(k1);
        if (at >= 0) {
          const int row = n % a.pages.size;
          T *kr = (T *)(a.pages.k.p + page_row(a.pages.k, at, row) + g * a.pages.k.head);
          T *vr = (T *)(a.pages.v.p + page_row(a.pages.v, at, row) + g * a.pages.v.head);
          const T *vs = (const T *)(a.v.p + b * a.v.batch + g * a.v.head);
          kr[i0] = k0;
          kr[i1] = k1;
          vr[2 * p] = vs[2 * p];
          vr[2 * p + 1] = vs[2 * p + 1];
        }
      } else {
        lds.q[hh][i0] = r0 * c;
        lds.q[hh][i1] = r1 * c;
      }
    }
    __syncthreads();
    const int m16 = lane & 15, u4 = lane >> 4;
    Pair<T> q[GP::NS];
#pragma unroll
    for (int s = 0; s < GP::NS; ++s) {
      const float *f = &lds.q[m16][(4 * s + u4) * GP::E];
      if constexpr (sizeof(T) == 2) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = f[i];
        q[s] = split8_any(w);
      } else {
        q[s].hi = *reinterpret_cast<const uint4 *>(f);
      }
    }

    State<T, DH> st;
    // the next group is on the way while this one is used, where the registers hold both (fp32 rows
    // of 512 bytes: 128 registers a group; the waves' loads keep the memory busy there)
    constexpr bool AHEAD = sizeof(T) * DH <= 256;
    // The wave's groups, x holding its first group of the cache if it has any, page what the next one's lanes look up.
    auto pass = [&](auto guard) {
      constexpr bool GUARD = decltype(guard)::value;
      st.clear();
      if (s0 + wave == 0) {  // the new token: a group of one key
        GP y;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int s = 0; s < GP::NS; ++s) {
            y.k[t][s] = make_uint4(0, 0, 0, 0);
            if (t == 0 && m16 == 0) {
              const float *f = &lds.q[16][(4 * s + u4) * GP::E];
              if constexpr (sizeof(T) == 2) {
                float w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = f[i];
                y.k[t][s] = split8(w).hi;
              } else {
                y.k[t][s] = *reinterpret_cast<const uint4 *>(f);
              }
            }
          }
        const char *vs = a.v.p + b * a.v.batch + g * a.v.head;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int w = 0; w < GP::VW; ++w) {
            const int d = m16 * GP::EV * (int)sizeof(T) + 4 * w;
            y.v[i][w] = i == 0 && u4 == 0 && d < a.hd * (int)sizeof(T) ? *(const uint32_t *)(vs + d) : 0u;
          }
        st.template add<GUARD>(y, q, [](int i) { return i < 1; }, lane);
      }
      for (int i = first; i < s1; i += WAVES) {
        const int next = i + WAVES;
        const uint32_t now = mask;
        if constexpr (AHEAD && !GUARD) {
          GP y;
          if (next < s1) {
            const int then = next + WAVES < s1 ? page_of(a, table, seen, next + WAVES, lane) : -1;
            mask = fetch(y, a, seen, g, next, page, lane);
            page = then;
          }
          st.template add<GUARD>(x, q, [=](int k) { return now >> k & 1u; }, lane);
          if (next < s1) x = y;
        } else {
          st.template add<GUARD>(x, q, [=](int k) { return now >> k & 1u; }, lane);
          if (next < s1) {
            const int then = next + WAVES < s1 ? page_of(a, table, seen, next + WAVES, lane) : -1;
            mask = fetch(x, a, seen, g, next, page, lane);
            page = then;
          }
        }
      }
    };
    pass(std::false_type());
    if constexpr (sizeof(T) == 2) {
      if (__builtin_expect(st.spoilt(), 0)) {
        if (first < s1) {
          mask = fetch(x, a, seen, g, first, page_of(a, table, seen, first, lane), lane);
          if (first + WAVES < s1) page = page_of(a, table, seen, first + WAVES, lane);
        }
        pass(std::true_type());
      }
    }

    // join the waves
    float l = half_sum(st.l);
    l += __shfl_xor(l, 16);
    if (u4 == 0) {
      lds.tops[wave][m16] = st.m;
      lds.tots[wave][m16] = l;
    }
    if (m16 < cols) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < GP::EV; j += 4)
          *reinterpret_cast<float4 *>(&lds.sums[(wave * cols + m16) * LD + GP::EV * (4 * u4 + r) + j]) =
              make_float4(st.acc[j][r], st.acc[j + 1][r], st.acc[j + 2][r], st.acc[j + 3][r]);
    }
    __syncthreads();
    const int wide = min(16, per);  // columns of a slot
    for (int i = tid; i < cols * a.hd; i += THREADS) {
      const int col = i / a.hd, d = i % a.hd;
      float top = lds.tops[0][col];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) top = fmaxf(top, lds.tops[w][col]);
      float s = 0.f, t = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float mw = lds.tops[w][col];
        const float f = mw == -INFINITY ? (lds.tots[w][col] == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(mw - top);
        s = __builtin_fmaf(f, lds.sums[(w * cols + col) * LD + d], s);
        t = __builtin_fmaf(f, lds.tots[w][col], t);
      }
      if (slot < 0) {
        *(T *)(a.o.p + b * a.o.batch + (e0 + col) * a.o.head + d * sizeof(T)) = from_f32<T>(quotient(s, t));
      } else {
        const int64_t row = (int64_t)slot * wide + col;
        a.part[row * a.hd + d] = s;
        if (d == 0) {
          float *ml = a.part + (int64_t)2 * a.blocks * wide * a.hd + row * 2;
          ml[0] = top;
          ml[1] = t;
        }
      }
    }
  }
};

__device__ __forceinline__ int columns(const PagedArgs &a) { return (a.H / a.G + 15) / 16; }

template <typename T>
__device__ __forceinline__ void write_zeros(const PagedArgs &a, int b, int e0, int cols, int tid, int threads) {
  for (int i = tid; i < cols * a.hd; i += threads)
    *(T *)(a.o.p + b * a.o.batch + (e0 + i / a.hd) * a.o.head + (i % a.hd) * sizeof(T)) = from_f32<T>(0.f);
}

// A block for a unit.
template <typename T, int DH, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 1) void attn_paged_kernel(PagedArgs a) {
  using S = Step<T, DH, WAVES>;
  extern __shared__ __align__(16) unsigned char raw[];
  typename S::Lds &lds = *(typename S::Lds *)raw;
  const int tid = threadIdx.x, b = blockIdx.y, g = blockIdx.x / columns(a), cb = blockIdx.x % columns(a);
  const int n = uniform(a.lengths[b]);
  if (n < 0 || n >= a.pages.capacity) {
    const int per = a.H / a.G;
    write_zeros<T>(a, b, g * per + cb * 16, min(16, per - cb * 16), tid, S::THREADS);
    return;
  }
  const Seen seen = seen_of(a.window, a.sinks, n);
  S::run(a, lds, b, seen, g, cb, 0, seen.groups, -1, tid);
}

// A block for an equal share of all groups, no less than two for each of its waves.
template <typename T, int DH, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 1) void attn_paged_flat_kernel(PagedArgs a) {
  using S = Step<T, DH, WAVES>;
  extern __shared__ __align__(16) unsigned char raw[];
  typename S::Lds &lds = *(typename S::Lds *)raw;
  __shared__ int64_t ends[kMostSeqs];  // groups of all units up to and with a sequence's
  __shared__ int64_t totals[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int units = a.G * columns(a);
  int64_t before = 0;
  for (int i0 = 0; i0 < a.B; i0 += S::THREADS) {
    const int i = i0 + tid, n = i < a.B ? a.lengths[i] : -1;
    int64_t sum = n >= 0 && n < a.pages.capacity ? (int64_t)seen_of(a.window, a.sinks, n).groups * units : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t x = __shfl_up((long long)sum, d);
      if (lane >= d) sum += x;
    }
    if (lane == 63) totals[wave] = sum;
    __syncthreads();
    sum += before;
    for (int w = 0; w < wave; ++w) sum += totals[w];
    if (i < a.B) ends[i] = sum;
    for (int w = 0; w < WAVES; ++w) before += totals[w];
    __syncthreads();
  }
  const int64_t all = before;
  const int64_t share = max((all + gridDim.x - 1) / gridDim.x, (int64_t)2 * WAVES);
  int64_t at = share * blockIdx.x;
  const int64_t stop = min(at + share, all);
  if (at >= stop) return;
  int b = 0, hi = a.B - 1;  // the first sequence that ends past `at`
  while (b < hi) {
    const int mid = (b + hi) >> 1;
    if (ends[mid] > at) hi = mid;
    else b = mid + 1;
  }
  b = uniform(b);
  while (at < stop) {
    while (ends[b] <= at) ++b;
    const Seen seen = seen_of(a.window, a.sinks, uniform(a.lengths[b]));
    const int64_t base = b > 0 ? ends[b - 1] : 0;
    const int unit = uniform((int)((at - base) / seen.groups));
    const int64_t first = base + (int64_t)unit * seen.groups;
    const int s0 = uniform((int)(at - first)), s1 = uniform((int)min((int64_t)seen.groups, stop - first));
    const int last = (int)((first + seen.groups - 1) / share);
    if (s0 == 0 && tid == 0) a.spans[(int64_t)b * units + unit] = make_int2(blockIdx.x, last);
    const int slot = s0 > 0 ? 2 * blockIdx.x : last > (int)blockIdx.x ? 2 * blockIdx.x + 1 : -1;
    S::run(a, lds, b, seen, unit / columns(a), unit % columns(a), s0, s1, slot, tid);
    at += s1 - s0;
  }
}

// o of the units that several blocks share, and of the slots without a sequence: a block for a query head.
constexpr int kJoinRows = 8;  // parts that are added at a time
template <typename T>
__global__ __launch_bounds__(kJoinRows * 32) void attn_paged_join_kernel(PagedArgs a) {
  __shared__ float4 sums[kJoinRows][32];
  __shared__ float most[kJoinRows * 32 / 64], tots[kJoinRows][32];
  const int tid = threadIdx.x, lane = tid & 63, e = blockIdx.x, b = blockIdx.y;
  const int per = a.H / a.G, g = e / per, cb = e % per / 16, col = e % per % 16, wide = min(16, per);
  const int n = a.lengths[b];
  if (n < 0 || n >= a.pages.capacity) {
    write_zeros<T>(a, b, e, 1, tid, kJoinRows * 32);
    return;
  }
  const int2 span = a.spans[(int64_t)b * a.G * columns(a) + g * columns(a) + cb];
  if (span.x == span.y) return;
  const int parts = span.y - span.x + 1;
  const float *ml = a.part + (int64_t)2 * a.blocks * wide * a.hd;
  auto row = [&](int i) { return (int64_t)(2 * (span.x + i) + (i == 0)) * wide + col; };
  float top = -INFINITY;
  for (int i = tid; i < parts; i += kJoinRows * 32) top = fmaxf(top, ml[2 * row(i)]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  if (lane == 0) most[tid >> 6] = top;
  __syncthreads();
  for (int w = 0; w < kJoinRows * 32 / 64; ++w) top = fmaxf(top, most[w]);
  const int quad = tid & 31, r = tid >> 5;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  float t = 0.f;
#pragma unroll 4
  for (int i = r; i < parts; i += kJoinRows) {
    const int64_t at = row(i);
    const float m = ml[2 * at], l = ml[2 * at + 1];
    const float f = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(m - top);
    t = __builtin_fmaf(f, l, t);
    if (4 * quad < a.hd) {
      const float4 x = *reinterpret_cast<const float4 *>(a.part + at * a.hd + 4 * quad);
      s.x = __builtin_fmaf(f, x.x, s.x);
      s.y = __builtin_fmaf(f, x.y, s.y);
      s.z = __builtin_fmaf(f, x.z, s.z);
      s.w = __builtin_fmaf(f, x.w, s.w);
    }
  }
  sums[r][quad] = s;
  tots[r][quad] = t;
  __syncthreads();
  if (r > 0 || 4 * quad >= a.hd) return;
#pragma unroll
  for (int i = 1; i < kJoinRows; ++i) {
    const float4 x = sums[i][quad];
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
    t += tots[i][quad];
  }
  T *o = (T *)(a.o.p + b * a.o.batch + e * a.o.head) + 4 * quad;
  o[0] = from_f32<T>(quotient(s.x, t));
  o[1] = from_f32<T>(quotient(s.y, t));
  o[2] = from_f32<T>(quotient(s.z, t));
  o[3] = from_f32<T>(quotient(s.w, t));
}

int64_t most_groups(const PagedArgs &a) {  // of a unit
  const int64_t seen = a.window ? std::min<int64_t>(a.pages.capacity, (int64_t)a.window + a.sinks + 2 * kGroup) : a.pages.capacity;
  return 1 + (seen + kGroup - 1) / kGroup;
}

template <typename T, int DH>
int launch(const PagedArgs &a, hipStream_t st) {
  constexpr int WAVES = 8;
  using S = Step<T, DH, WAVES>;
  const int per = a.H / a.G, units = a.G * ((per + 15) / 16);
  const size_t lds = S::lds_bytes(std::min(16, per));
  if (a.blocks == 0) {
    attn_paged_kernel<T, DH, WAVES><<<dim3(units, a.B), dim3(S::THREADS), lds, st>>>(a);
    return DYNCONV_OK;
  }
  attn_paged_flat_kernel<T, DH, WAVES><<<dim3(a.blocks), dim3(S::THREADS), lds, st>>>(a);
  attn_paged_join_kernel<T><<<dim3(a.H, a.B), dim3(kJoinRows * 32), 0, st>>>(a);
  return DYNCONV_OK;
}

}  // namespace

// Blocks of the flattened launch; 0 where a block reads the most that a sequence can have in a few steps, or the batch is large.
int paged_blocks(const PagedArgs &a) {
  const int64_t units = (int64_t)a.B * a.G * ((a.H / a.G + 15) / 16), most = most_groups(a);
  if (most <= 33 || a.B > kMostSeqs) return 0;
  return (int)std::min<int64_t>(512, (units * most + 15) / 16);
}

int64_t paged_workspace(const PagedArgs &a) {
  const int64_t n = paged_blocks(a), wide = std::min(16, a.H / a.G);
  if (n == 0) return 0;
  const int64_t units = (int64_t)a.B * a.G * ((a.H / a.G + 15) / 16);
  return 2 * n * wide * (a.hd + 2) * 4 + units * 8;
}

int attn_paged(const PagedArgs &a, int dtype, hipStream_t st) {
  if (dtype == DYNCONV_BF16) return a.hd <= 64 ? launch<bf16, 64>(a, st) : launch<bf16, 128>(a, st);
  return a.hd <= 64 ? launch<float, 64>(a, st) : launch<float, 128>(a, st);
}

}  // namespace dynconv
