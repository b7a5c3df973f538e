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
// Lengths differ, and the host does not know them.  Where a block reads the most that a sequence can have in a few steps it takes
// a unit whole, its waves every eighth group.  Otherwise the launch is flat: the groups of all sequences stand in one row, of which
// each block finds its equal share from the lengths (a sum over the batch in LDS) and takes the sequences that lie in it one
// after another, a wave for each of as many key/value heads: they read the rows of a token side by side, and
// no wave waits for another.  Sequences that several blocks share are joined by a second kernel, in the order of the blocks.
//
// bf16, 16 + 4 heads of 128: 64 sequences of up to 8191 tokens (614 MB) 118 us, 5.3 TB/s, the join 10 of them; 64 windows of 1024
// (131 MB) 29 us; one sequence of 131071 (268 MB) 59 us, the join 9; 12 heads of 64, one sequence of 1024 (3 MB) 11 us, a chain
// of length, pages, rows, join of the waves.
#include <algorithm>
#include <type_traits>

#include "attn_group.h"
#include "attn_paged.h"
#include "kernels.h"
#include "rope.h"

namespace dynconv {

namespace {

constexpr int kMostSeqs = 1024;   // whose lengths a block of the flat launch adds up
// of the flat launch: with 4 key/value heads side by side a block of four for each CU (64 sequences of up to 8191 tokens, 16 + 4 heads
// of 128: 119 us; 2048: 121, 4096: 135; blocks of one wave instead of side by side: 140).  With 6 heads and more blocks are of
// 6 to 8 waves and fewer than the CUs: 24 + 6 heads 220 us, 32 + 8 328, 16 + 16 604, 4.2, 3.8 and 4.1 TB/s against 5.3.
constexpr int kFlatWaves = 1024;

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
      const u32x4 w = __builtin_nontemporal_load((Global16)(chunk * G::E < a.hd ? row + chunk * 16 : zero));
      x.k[t][i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const char *row = from_lane(vr, 8 * u + i);
    if constexpr (G::VW == 2) {
      const u32x2 w = __builtin_nontemporal_load((Global8)(m * G::EV < a.hd ? row + m * G::EV * (int)sizeof(T) : zero));
      x.v[i][0] = w[0];
      x.v[i][1] = w[1];
    } else {
#pragma unroll
      for (int j = 0; j < G::VW / 4; ++j) {
        const u32x4 w = __builtin_nontemporal_load((Global16)(m * G::EV + j * G::E < a.hd ? row + m * G::EV * (int)sizeof(T) + 16 * j : zero));
#pragma unroll
        for (int c = 0; c < 4; ++c) x.v[i][4 * j + c] = w[c];
      }
    }
  }
  return mask;
}

// The columns' operand in LDS: with two groups of rows in registers there is no room for it there (heads of 128).
template <typename T>
struct Columns {
  static constexpr int PARTS = sizeof(T) == 2 ? 2 : 1;
  const uint4 *p;  // [step][part][lane]
  __device__ __forceinline__ Pair<T> operator[](int i) const {
    Pair<T> x;
    x.hi = p[i * PARTS * 64];
    if constexpr (PARTS == 2) x.lo = p[i * 2 * 64 + 64];
    return x;
  }
};

// Groups s0 .. s1 - 1 of a unit: sequence b, key/value head g, column block cb.
struct Part {
  Seen seen;
  int b, g, cb, s0, s1;
};

__device__ __forceinline__ int columns(const PagedArgs &a) { return (a.H / a.G + 15) / 16; }

// Waits for a group.  The next one is sent for when this one has come and not before: two on their way for each of a CU's
// eight waves (32 KB, heads of 128 in bf16) are more than its share of the caches between it and the memory, and lines are
// fetched again (a kernel that reads such rows alone: 6.8 TB/s with 8 to 24 KB on their way for a wave, 4.2 with 32).
template <typename T, int DH>
__device__ __forceinline__ void here(Group<T, DH> &x) {
#pragma unroll
  for (int t = 0; t < 2; ++t) arrived(x.k[t]);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int w = 0; w < Group<T, DH>::VW; ++w) asm volatile("" : "+v"(x.v[i][w]));
}

// A wave's work on parts, every STRIDE-th group of which is its own.
template <typename T, int DH>
struct Wave {
  static constexpr int LD = DH + 4;  // (rows shifted by 16 bytes against bank conflicts)
  // the next group is on the way while this one is used, where the registers hold both (fp32 rows
  // of 512 bytes: 128 registers a group; the waves' loads keep the memory busy there)
  static constexpr bool AHEAD = sizeof(T) * DH <= 256;
  using GP = Group<T, DH>;
  static constexpr int OPERAND = GP::NS * Columns<T>::PARTS * 64;  // vectors of 16 bytes
  // in LDS, for `wide` columns: the columns' operand, then the query heads times scale log2 e and the new key
  static __host__ __device__ int lds_bytes(int wide) { return OPERAND * 16 + (wide + 1) * LD * 4; }

  const PagedArgs &a;
  uint4 *operand;
  float *qs;
  int lane, wide;
  // what is on its way: the wave's next group, which of its keys there are, and the pages of the one after it; and of the part
  // that was asked for the pages of its first two groups
  GP x;
  uint32_t mask;
  int page, ahead[2];
  State<T, DH> st;

  __device__ __forceinline__ Wave(const PagedArgs &args, unsigned char *lds, int l) : a(args), lane(l) {
    wide = min(16, a.H / a.G);
    operand = (uint4 *)lds;
    qs = (float *)(operand + OPERAND);
  }
  __device__ __forceinline__ int columns_of(const Part &p) const { return min(16, a.H / a.G - p.cb * 16); }
  __device__ __forceinline__ int first_head(const Part &p) const { return p.g * (a.H / a.G) + p.cb * 16; }
  __device__ __forceinline__ const int32_t *table(const Part &p) const { return a.pages.table + p.b * a.pages.table_row; }
  // (the new token is no group of the cache)
  __device__ __forceinline__ int first_group(int at, int stride) const { return at == 0 ? stride : at; }

  // Asks for the pages of the first groups from `at` on.
  __device__ __forceinline__ void ask(const Part &p, int at, int stride) {
    const int first = first_group(at, stride);
    ahead[0] = first < p.s1 ? page_of(a, table(p), p.seen, first, lane) : -1;
    ahead[1] = first + stride < p.s1 ? page_of(a, table(p), p.seen, first + stride, lane) : -1;
  }
  // Sends for the rows of the first one.
  __device__ __forceinline__ void send(const Part &p, int at, int stride) {
    const int first = first_group(at, stride);
    if (first < p.s1) mask = fetch(x, a, p.seen, p.g, first, ahead[0], lane);
    page = ahead[1];
  }

  // q and the new key, turned, in LDS, `sharers` waves taking part (this one is the i-th); the new key and value into their
  // page.  A lane has one pair of the heads: its angle is formed once.  The first head's pair and the frequency are sent for ahead of
  // the rows (loads come back in the order they were sent).
  struct Pair0 {
    double freq;
    float u, w;
  };
  __device__ __forceinline__ const T *pair_source(const Part &p, int h) const {
    return (const T *)(h == columns_of(p) ? a.k.p + p.b * a.k.batch + p.g * a.k.head
                                          : a.q.p + p.b * a.q.batch + (first_head(p) + h) * a.q.head);
  }
  // Elements of pair m: halves or neighbours.
  __device__ __forceinline__ int low(int m) const { return m < a.rot / 2 && !a.interleaved ? m : 2 * m; }
  __device__ __forceinline__ int high(int m) const { return m < a.rot / 2 && !a.interleaved ? m + a.rot / 2 : 2 * m + 1; }
  __device__ __forceinline__ Pair0 ask_pair(const Part &p, int i) const {
    const int half = a.hd / 2, abreast = 64 / half, m = lane % half, h = i * abreast + lane / half;
    Pair0 x = {0.0, 0.f, 0.f};
    if (lane / half >= abreast || h > columns_of(p)) return x;
    const T *src = pair_source(p, h);
    if (m < a.rot / 2) x.freq = a.freqs[m];
    x.u = to_f32(src[low(m)]);  // (rot is even: the rest starts at 2 (rot/2))
    x.w = to_f32(src[high(m)]);
    return x;
  }
  __device__ __forceinline__ void turn_pairs(const Part &p, Pair0 x, int i, int sharers) {
    const int half = a.hd / 2, abreast = 64 / half, m = lane % half, cols = columns_of(p), n = p.seen.n;
    const bool turned = m < a.rot / 2;
    const int i0 = low(m), i1 = high(m);
    float cs = 1.f, sn = 0.f;
    if (turned) {
      turn(n, x.freq, cs, sn);
      cs *= a.factor;
      sn *= a.factor;
    }
    const float c = a.scale * kLog2e;
    const int first = i * abreast + lane / half;
    if (lane / half >= abreast) return;
#pragma unroll 4
    for (int h = first; h <= cols; h += sharers * abreast) {
      float u = x.u, w = x.w;
      if (h != first) {
        const T *src = pair_source(p, h);
        u = to_f32(src[i0]);
        w = to_f32(src[i1]);
      }
      float r0 = u, r1 = w;
      if (turned) turn_pair(u, w, cs, sn, r0, r1);
      float *to = qs + (h == cols ? wide : h) * LD;
      if (h == cols) {
        r0 = to_f32(from_f32<T>(r0));
        r1 = to_f32(from_f32<T>(r1));
      } else {
        r0 *= c;
        r1 *= c;
      }
      to[i0] = r0;
      to[i1] = r1;
      if (h == cols && p.s0 == 0 && p.cb == 0) {
        const int at = page_at(table(p), a.pages.size, a.pages.n_pages, n), row = n % a.pages.size;
        if (at >= 0) {
          T *kr = (T *)(a.pages.k.p + page_row(a.pages.k, at, row) + p.g * a.pages.k.head);
          T *vr = (T *)(a.pages.v.p + page_row(a.pages.v, at, row) + p.g * a.pages.v.head);
          const T *vs = (const T *)(a.v.p + p.b * a.v.batch + p.g * a.v.head);
          kr[i0] = from_f32<T>(r0);
          kr[i1] = from_f32<T>(r1);
          vr[2 * m] = vs[2 * m];
          vr[2 * m + 1] = vs[2 * m + 1];
        }
      }
    }
  }
  // The columns' operand from it.
  __device__ __forceinline__ void build(int cols, int i, int sharers) {
    for (int s = i; s < GP::NS; s += sharers) {
      const int chunk = 4 * s + (lane >> 4);
      const float *from = qs + (lane & 15) * LD + chunk * GP::E;
      float f[GP::E];
#pragma unroll
      for (int j = 0; j < GP::E; ++j) f[j] = (lane & 15) < cols && chunk * GP::E < a.hd ? from[j] : 0.f;
      if constexpr (sizeof(T) == 2) {
        const Pair<T> c = split8_any(f);
        operand[2 * s * 64 + lane] = c.hi;
        operand[(2 * s + 1) * 64 + lane] = c.lo;
      } else {
        operand[s * 64 + lane] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      }
    }
  }

  // The wave's groups from `at` on; x, mask and page as send() left them.
  template <bool GUARD>
  __device__ __forceinline__ void pass(const Part &p, int at, int stride) {
    const int m16 = lane & 15, u4 = lane >> 4;
    const Columns<T> q = {operand + lane};
    st.clear();
    if (at == 0) {  // the new token: a group of one key
      const float *key = qs + wide * LD;
      const char *vs = a.v.p + p.b * a.v.batch + p.g * a.v.head;
      GP y;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int s = 0; s < GP::NS; ++s) {
          const int chunk = 4 * s + u4;
          y.k[t][s] = make_uint4(0, 0, 0, 0);
          if (t == 0 && m16 == 0 && chunk * GP::E < a.hd) {
            const float *f = key + chunk * GP::E;
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
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int w = 0; w < GP::VW; ++w) {
          const int d = m16 * GP::EV * (int)sizeof(T) + 4 * w;
          y.v[i][w] = i == 0 && u4 == 0 && d < a.hd * (int)sizeof(T) ? *(const uint32_t *)(vs + d) : 0u;
        }
      st.template add<GUARD>(y, q, [](int i) { return i < 1; }, lane);
    }
    for (int i = first_group(at, stride); i < p.s1; i += stride) {
      const int next = i + stride;
      const uint32_t now = mask;
      asm volatile("" ::: "memory");  // (q is read again for each group)
      if constexpr (AHEAD && !GUARD) {
        GP y;
        here(x);
        if (next < p.s1) {
          const int then = next + stride < p.s1 ? page_of(a, table(p), p.seen, next + stride, lane) : -1;
          mask = fetch(y, a, p.seen, p.g, next, page, lane);
          page = then;
        }
        st.template add<GUARD>(x, q, [=](int k) { return now >> k & 1u; }, lane);
        if (next < p.s1) x = y;
      } else {
        st.template add<GUARD>(x, q, [=](int k) { return now >> k & 1u; }, lane);
        if (next < p.s1) {
          const int then = next + stride < p.s1 ? page_of(a, table(p), p.seen, next + stride, lane) : -1;
          mask = fetch(x, a, p.seen, p.g, next, page, lane);
          page = then;
        }
      }
    }
  }
  __device__ __forceinline__ void sum(const Part &p, int at, int stride) {
    pass<false>(p, at, stride);
    if constexpr (sizeof(T) == 2) {
      if (__builtin_expect(st.spoilt(), 0)) {
        const int next[2] = {ahead[0], ahead[1]};  // (of the part that was asked for after this one)
        ask(p, at, stride);
        send(p, at, stride);
        pass<true>(p, at, stride);
        ahead[0] = next[0];
        ahead[1] = next[1];
      }
    }
  }
  // The sum of the wave's weights, in all lanes of a column.
  __device__ __forceinline__ float total() const {
    const float l = half_sum(st.l);
    return l + __shfl_xor(l, 16);
  }
};

// A block for a unit, its waves every eighth group.
constexpr int kWaves = 8;
template <typename T, int DH>
__global__ __launch_bounds__(kWaves * 64, 2) void attn_paged_kernel(PagedArgs a) {
  using W = Wave<T, DH>;
  constexpr int THREADS = kWaves * 64, LD = W::LD;
  extern __shared__ __align__(16) unsigned char raw[];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), b = blockIdx.y, g = blockIdx.x / columns(a);
  const int n = uniform(a.lengths[b]);
  Part p = {seen_of(a.window, a.sinks, n), b, g, (int)blockIdx.x % columns(a), 0, 0};
  W w(a, raw, tid & 63);
  const int cols = w.columns_of(p), e0 = w.first_head(p);
  if (n < 0 || n >= a.pages.capacity) {
    for (int i = tid; i < cols * a.hd; i += THREADS)
      *(T *)(a.o.p + b * a.o.batch + (e0 + i / a.hd) * a.o.head + (i % a.hd) * sizeof(T)) = from_f32<T>(0.f);
    return;
  }
  p.s1 = p.seen.groups;
  w.ask(p, wave, kWaves);
  const typename W::Pair0 pair = w.ask_pair(p, wave);
  w.send(p, wave, kWaves);
  w.turn_pairs(p, pair, wave, kWaves);
  __syncthreads();
  w.build(cols, wave, kWaves);
  __syncthreads();
  w.sum(p, wave, kWaves);

  // join the waves
  float *sums = (float *)(raw + W::lds_bytes(w.wide)), *stats = sums + kWaves * cols * LD;
  const int m16 = tid & 15, u4 = (tid & 63) >> 4;
  const float l = w.total();
  if (m16 < cols) {
    if (u4 == 0) {
      stats[(wave * cols + m16) * 2] = w.st.m;
      stats[(wave * cols + m16) * 2 + 1] = l;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < W::GP::EV; j += 4)
        *reinterpret_cast<float4 *>(&sums[(wave * cols + m16) * LD + W::GP::EV * (4 * u4 + r) + j]) =
            make_float4(w.st.acc[j][r], w.st.acc[j + 1][r], w.st.acc[j + 2][r], w.st.acc[j + 3][r]);
  }
  __syncthreads();
  for (int i = tid; i < cols * a.hd; i += THREADS) {
    const int col = i / a.hd, d = i - col * a.hd;
    float top = stats[col * 2];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) top = fmaxf(top, stats[(k * cols + col) * 2]);
    float s = 0.f, t = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      const float m = stats[(k * cols + col) * 2], l = stats[(k * cols + col) * 2 + 1];
      const float f = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(m - top);
      s = __builtin_fmaf(f, sums[(k * cols + col) * LD + d], s);
      t = __builtin_fmaf(f, l, t);
    }
    *(T *)(a.o.p + b * a.o.batch + (e0 + col) * a.o.head + d * sizeof(T)) = from_f32<T>(quotient(s, t));
  }
}

// A block of a.abreast waves, one for each of as many units of a sequence, for an equal share of all groups, no less than kLeast.
constexpr int kLeast = 4;
template <typename T, int DH>
__global__ __launch_bounds__(512, 2) void attn_paged_flat_kernel(PagedArgs a) {
  using W = Wave<T, DH>;
  extern __shared__ __align__(16) unsigned char raw[];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int units = a.G * columns(a), sets = units / a.abreast, wide = min(16, a.H / a.G);
  int *ends = (int *)(raw + a.abreast * W::lds_bytes(wide));  // groups of all sets of units up to and with a sequence's
  int all = 0;
  for (int i0 = 0; i0 < a.B; i0 += 64) {  // (every wave for itself, to the same numbers)
    const int i = i0 + lane, n = i < a.B ? a.lengths[i] : -1;
    int sum = n >= 0 && n < a.pages.capacity ? seen_of(a.window, a.sinks, n).groups * sets : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int x = __shfl_up(sum, d);
      if (lane >= d) sum += x;
    }
    sum += all;
    if (i < a.B) ends[i] = sum;
    all = __builtin_amdgcn_readlane(sum, 63);
  }
  wave_sync();
  const int share = max((int)(((uint32_t)all + gridDim.x - 1) / gridDim.x), kLeast);
  if (all == 0 || blockIdx.x > (uint32_t)(all - 1) / (uint32_t)share) return;
  int at = share * blockIdx.x;
  const int stop = (int)min((uint32_t)at + (uint32_t)share, (uint32_t)all);
  int b = 0, hi = a.B - 1;  // the first sequence that ends past `at`
  while (b < hi) {
    const int mid = (b + hi) >> 1;
    if (uniform(ends[mid]) > at) hi = mid;
    else b = mid + 1;
  }
  // The part that begins at `at`, which moves on to its end; slot: where its sums go, -1: it is a whole unit.
  auto next_part = [&](int &slot) {
    Part p;
    while (uniform(ends[b]) <= at) ++b;
    p.seen = seen_of(a.window, a.sinks, uniform(a.lengths[b]));
    p.b = b;
    const int base = b > 0 ? uniform(ends[b - 1]) : 0;
    const int set = uniform((uint32_t)(at - base) / (uint32_t)p.seen.groups), first = base + set * p.seen.groups;
    const int unit = set * a.abreast + wave;
    p.g = unit / columns(a);
    p.cb = unit - p.g * columns(a);
    p.s0 = at - first;
    p.s1 = min(p.seen.groups, stop - first);
    const int last = uniform((uint32_t)(first + p.seen.groups - 1) / (uint32_t)share);
    if (p.s0 == 0 && lane == 0) a.spans[(int64_t)b * units + unit] = make_int2(blockIdx.x, last);
    slot = p.s0 > 0 ? 2 * blockIdx.x : last > (int)blockIdx.x ? 2 * blockIdx.x + 1 : -1;
    at = first + p.s1;
    return p;
  };
  W w(a, raw + wave * W::lds_bytes(wide), lane);
  const int m16 = lane & 15, u4 = lane >> 4;
  int slot, next_slot = 0;
  Part p = next_part(slot), q;
  w.ask(p, p.s0, 1);
  w.send(p, p.s0, 1);
  while (true) {
    const int cols = w.columns_of(p);
    w.turn_pairs(p, w.ask_pair(p, 0), 0, 1);
    wave_sync();
    w.build(cols, 0, 1);
    wave_sync();
    const bool more = at < stop;
    if (more) {
      q = next_part(next_slot);
      w.ask(q, q.s0, 1);
    }
    w.sum(p, p.s0, 1);
    if (more) w.send(q, q.s0, 1);  // (while the sums are written)
    const float l = w.total();
    if (m16 < cols) {
      const bool none = l == 0.f;  // (as in quotient: whatever the values without a weight hold)
      const float inv = none ? 0.f : 1.f / l;
      const int e = w.first_head(p) + m16;
      const int64_t row = ((int64_t)slot * a.abreast + wave) * wide + m16;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = W::GP::EV * (4 * u4 + r);
        if (slot < 0) {
          T *o = (T *)(a.o.p + p.b * a.o.batch + e * a.o.head) + d;
#pragma unroll
          for (int j = 0; j < W::GP::EV; ++j)
            if (d + j < a.hd) o[j] = from_f32<T>(none ? 0.f : w.st.acc[j][r] * inv);
        } else {
          float *o = a.part + row * a.hd + d;
#pragma unroll
          for (int j = 0; j < W::GP::EV; j += 4)
            if (d + j < a.hd)
              *reinterpret_cast<float4 *>(o + j) = make_float4(w.st.acc[j][r], w.st.acc[j + 1][r], w.st.acc[j + 2][r], w.st.acc[j + 3][r]);
        }
      }
      if (slot >= 0 && u4 == 0) {
        float *ml = a.part + (int64_t)2 * a.blocks * a.abreast * wide * a.hd;
        ml[row * 2] = w.st.m;
        ml[row * 2 + 1] = l;
      }
    }
    if (!more) break;
    p = q;
    slot = next_slot;
  }
}

// o of the units that several blocks share, and of the slots without a sequence: a block for 32 elements of a query head.
constexpr int kJoinRows = 32;  // parts that are added at a time, by 8 threads each
template <typename T>
__global__ __launch_bounds__(kJoinRows * 8) void attn_paged_join_kernel(PagedArgs a) {
  __shared__ float4 sums[kJoinRows][8];
  __shared__ float most[kJoinRows / 8], tots[kJoinRows];
  const int pieces = (a.hd + 31) / 32;
  const int tid = threadIdx.x, lane = tid & 63, e = blockIdx.x / pieces, b = blockIdx.y;
  const int per = a.H / a.G, g = e / per, cb = e % per / 16, col = e % per % 16, wide = min(16, per);
  const int quad = tid & 7, r = tid >> 3, d = blockIdx.x % pieces * 32 + 4 * quad;
  T *o = (T *)(a.o.p + b * a.o.batch + e * a.o.head) + d;
  const int n = a.lengths[b];
  const bool idle = n < 0 || n >= a.pages.capacity;
  const int2 span = idle ? make_int2(0, 0) : a.spans[(int64_t)b * a.G * columns(a) + g * columns(a) + cb];
  if (span.x == span.y) {
    if (idle && r == 0 && d < a.hd)
      for (int i = 0; i < 4; ++i) o[i] = from_f32<T>(0.f);
    return;
  }
  const int parts = span.y - span.x + 1;
  const float *ml = a.part + (int64_t)2 * a.blocks * a.abreast * wide * a.hd;
  const int unit = g * columns(a) + cb;
  auto row = [&](int i) { return ((int64_t)(2 * (span.x + i) + (i == 0)) * a.abreast + unit % a.abreast) * wide + col; };
  float top = -INFINITY;
  for (int i = tid; i < parts; i += kJoinRows * 8) top = fmaxf(top, ml[2 * row(i)]);
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
  if (lane == 0) most[tid >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinRows / 8; ++w) top = fmaxf(top, most[w]);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  float t = 0.f;
#pragma unroll 4
  for (int i = r; i < parts; i += kJoinRows) {
    const int64_t at = row(i);
    const float m = ml[2 * at], l = ml[2 * at + 1];
    const float f = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(m - top);
    t = __builtin_fmaf(f, l, t);
    if (d < a.hd) {
      const float4 x = *reinterpret_cast<const float4 *>(a.part + at * a.hd + d);
      s.x = __builtin_fmaf(f, x.x, s.x);
      s.y = __builtin_fmaf(f, x.y, s.y);
      s.z = __builtin_fmaf(f, x.z, s.z);
      s.w = __builtin_fmaf(f, x.w, s.w);
    }
  }
  sums[r][quad] = s;
  if (quad == 0) tots[r] = t;
  __syncthreads();
  if (r > 0 || d >= a.hd) return;
  t = tots[0];
#pragma unroll
  for (int i = 1; i < kJoinRows; ++i) {
    const float4 x = sums[i][quad];
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
    t += tots[i];
  }
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
  using W = Wave<T, DH>;
  const int wide = std::min(16, a.H / a.G), units = a.G * ((a.H / a.G + 15) / 16);
  if (a.blocks == 0) {
    const int lds = W::lds_bytes(wide) + kWaves * wide * (W::LD + 2) * 4;
    attn_paged_kernel<T, DH><<<dim3(units, a.B), dim3(kWaves * 64), lds, st>>>(a);
    return DYNCONV_OK;
  }
  const int lds = a.abreast * W::lds_bytes(wide) + a.B * 4;
  attn_paged_flat_kernel<T, DH><<<dim3(a.blocks), dim3(a.abreast * 64), lds, st>>>(a);
  attn_paged_join_kernel<T><<<dim3(a.H * ((a.hd + 31) / 32), a.B), dim3(kJoinRows * 8), 0, st>>>(a);
  return DYNCONV_OK;
}

int units_of(const PagedArgs &a) { return a.G * ((a.H / a.G + 15) / 16); }

}  // namespace

// Units that a block of the flat launch takes side by side.
int paged_abreast(const PagedArgs &a) {
  int n = std::min(8, units_of(a));
  while (units_of(a) % n != 0) --n;
  return n;
}

// Blocks of the flat launch; 0 where a block reads the most that a sequence can have in a few steps, or the batch is large.
// A unit whole and flat, us, bf16: 64 windows of 1024, 16 + 4 heads of 128, 29 and 45; one sequence of 1024, 12 heads of 64, 12
// and 21; 64 sequences of up to 4095, 16 + 4 heads of 128, 84 and 74.  What a sequence can have is what the rule knows: one of 1024
// tokens in a table of 8192 takes the flat launch too, 20 us.
int paged_blocks(const PagedArgs &a) {
  const int64_t units = (int64_t)a.B * units_of(a), most = most_groups(a);
  if (most <= 96 || a.B > kMostSeqs || units * most >= (int64_t)1 << 31) return 0;
  return (int)std::min<int64_t>(kFlatWaves / paged_abreast(a), (units / paged_abreast(a) * most + kLeast - 1) / kLeast);
}

int64_t paged_workspace(const PagedArgs &a) {
  const int64_t n = paged_blocks(a), wide = std::min(16, a.H / a.G);
  if (n == 0) return 0;
  return 2 * n * paged_abreast(a) * wide * (a.hd + 2) * 4 + (int64_t)a.B * units_of(a) * 8;
}

int attn_paged(const PagedArgs &a, int dtype, hipStream_t st) {
  if (dtype == DYNCONV_BF16) return a.hd <= 64 ? launch<bf16, 64>(a, st) : launch<bf16, 128>(a, st);
  return a.hd <= 64 ? launch<float, 64>(a, st) : launch<float, 128>(a, st);
}

}  // namespace dynconv
