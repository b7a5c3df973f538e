// attn.h -- internal pieces of libdynconv's attention kernels: arguments,
// document bounds, LDS tiles and matrix-core fragments (attn_fwd.hip,
// attn_bwd.h).
//
// All three attention kernels have the same form.  A wave owns 32 rows (the
// queries in the forward and in dq, the keys in dk/dv), one per lane column;
// the rows of the other side stream through LDS in tiles.  Scores are formed
// with the streamed rows as the A operand, so D[streamed row][owned row] puts
// one owned row in each lane pair (l, l + 32): softmax statistics are lane
// scalars, and a second product that sums over the streamed rows takes its B
// operand from the very registers that hold the scores, because the order of
// a product's summed index is free as long as the A operand (read from LDS
// by columns) follows it.
#pragma once

#include "bufio.h"
#include "docs.h"
#include "mfma.h"

namespace dynconv {

struct AttnView {  // strides in bytes
  char *p;
  int64_t batch, row, head;
};

struct AttnArgs {
  AttnView q, k, v, o;
  AttnView d_o, dq, dk, dv;  // backward
  float *lse;                // [B, H, T]
  float *delta;              // backward workspace: do . o, [B, H, T]
  float *part;               // backward workspace: dk / dv of the splits of a group (n_split > 1)
  int B, T, H, G, hd;
  int n_split;  // dk/dv: blocks that share the queries of a tile of keys
  float scale;
  const int32_t *cu;
  int n_seqs;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 16 bytes of T as fp32 values (8 bf16 or 4 floats).
template <typename T>
__device__ __forceinline__ void widen(const uint4 &r, float (&f)[16 / sizeof(T)]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(w[i]);
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// The key from which on every row of a wave (queries qw .. qw+31, start: the lane's) sees
// keys, so that tiles from there on to the diagonal need no mask.  Rows of no document are
// let along: whatever they sum is not written.
__device__ __forceinline__ int full_from(int start, int qw, int limit) {
  return __builtin_amdgcn_readlane(start, __builtin_amdgcn_readfirstlane(min(31, max(0, limit - 1 - qw))));
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The other half wave's value (lane l ^ 32).
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// D[32x32] += A B over one step of the summed index: 16 (bf16) or 8 (fp32)
// values, of which a lane of half h = l / 32 holds one 16-byte chunk.
template <typename T>
__device__ __forceinline__ void mma_step(const uint4 &a, const uint4 &b, f32x16 &c) {
  if constexpr (sizeof(T) == 2) {
    c = mfma32(as_bf16x8(a), as_bf16x8(b), c);
  } else {
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  }
}

// A tile of rows of DH elements in LDS, row-major with gaps, so that modulo the 256 bytes of
// the banks the four rows of a group start 64 bytes apart (in some order), which the transposing
// reads need (4 rows x 64 bytes for a half wave), and 16 consecutive rows in 16 different
// places, which the reads by rows need (one 16-byte chunk each): a row takes an odd number of
// 64-byte pieces and a group of four an odd number of chunks.  Gaps and not a permutation of the
// chunks: every read of a tile is one lane address plus a constant (an XOR took 24 registers
// and as many adds a tile).
template <typename T, int DH>
struct Tile {
  static constexpr int E = 16 / (int)sizeof(T);  // elements of a chunk
  static constexpr int NC = DH / E;              // chunks of a row
  static constexpr int ROW = (NC / 4 | 1) * 64;  // bytes from row to row
  static constexpr int FOUR = ((3 * ROW / 16 + NC) | 1) * 16;  // from group to group
  static_assert(NC % 4 == 0, "");
  static constexpr int KS = NC / 2;              // steps of a sum over DH
  static constexpr int PS = 32 / (2 * E);        // steps of a sum over 32 rows
  static constexpr int ND = DH / 32;

  static constexpr int bytes(int rows) { return rows / 4 * FOUR; }
  static __device__ __forceinline__ int at(int r, int chunk) { return (r >> 2) * FOUR + (r & 3) * ROW + (chunk << 4); }

  // rows r0 .. r0+31, step s of the sum over DH: lane l holds chunk 2s + l/32 of row l%32
  static __device__ __forceinline__ uint4 rows(const unsigned char *t, int r0, int s, int lane) {
    return *reinterpret_cast<const uint4 *>(t + at(lane & 31, lane >> 5) + r0 / 4 * FOUR + s * 32);
  }
  // columns 32d .. 32d+31, step s of the sum over rows r0 .. r0+31, in the order in
  // which a score register block holds them: lane l, column l%32, half h = l/32:
  //   bf16: rows 16s + 8(i/4) + 4h + i%4, i = 0..7     fp32: rows 8s + 4h + i, i = 0..3
  static __device__ __forceinline__ uint4 cols(const unsigned char *t, int r0, int s, int d, int lane) {
    const int h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
      const unsigned char *p = t + at(4 * h + ((lane & 15) >> 2), ((lane >> 3) & 2) + ((lane >> 1) & 1)) + ((lane & 1) << 3) +
                               (r0 / 4 + 4 * s) * FOUR + d * 64;
      const uint2 lo = read_tr16(p), hi = read_tr16(p + 2 * FOUR);
      return make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      const unsigned char *p = t + at(4 * h, 0) + ((lane & 31) << 2) + (r0 / 4 + 2 * s) * FOUR + d * 128;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t *>(p + i * ROW);
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

// Score registers as the B operand of a sum over the streamed rows, step s
// (rounded to bf16 to nearest even for the bf16 matrix cores).
template <typename T>
__device__ __forceinline__ uint4 score_frag(const f32x16 &p, int s) {
  if constexpr (sizeof(T) == 2) {
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (bf16)p[8 * s + i];
    return __builtin_bit_cast(uint4, r);
  } else {
    return make_uint4(__float_as_uint(p[4 * s]), __float_as_uint(p[4 * s + 1]), __float_as_uint(p[4 * s + 2]),
                      __float_as_uint(p[4 * s + 3]));
  }
}
// streamed row (of 32) that register i of a score block holds in half h
__device__ __forceinline__ int score_row(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// Copies rows [row0, row0 + ROWS) of one head into a tile, through registers:
// fetch() issues the loads, store() writes what came.  Rows at or past `limit`
// and elements past head_dim come as zeros (of rows that overlap each other in
// memory, rows past `limit` come as whatever rows before it hold; nothing depends on them):
// the buffer ends with row limit - 1, so a load is one address sum.
template <typename T, int DH, int ROWS, int THREADS>
struct Stage {
  using TL = Tile<T, DH>;
  // lanes of a row: its chunks, or the next power of two (the lanes past them idle)
  static constexpr int W = TL::NC <= 8 ? 8 : TL::NC <= 16 ? 16 : 32;
  static constexpr int N = ROWS * W / THREADS, R = THREADS / W;  // loads of a thread, rows from one to the next
  static_assert(ROWS * W % THREADS == 0 && THREADS % W == 0 && TL::NC <= W, "");
  static_assert(R % 4 == 0 || R == 2, "");  // (whole groups of four, or half a group)
  uint4 r[N];
  __device__ __forceinline__ void fetch(const char *head, int64_t row_bytes, int row0, int limit, int hd, int tid) {
    const __amdgpu_buffer_rsrc_t rs =
        make_rsrc(head + (int64_t)row0 * row_bytes, rows_extent(row0, limit, row_bytes, hd * (int)sizeof(T), kOutside));
    const int chunk = tid % W;
    const uint32_t at = chunk * TL::E < hd ? (uint32_t)(tid / W) * (uint32_t)row_bytes + chunk * 16u : kOutside;
    const uint32_t step = (uint32_t)R * (uint32_t)row_bytes;
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = buf_load16(rs, at + i * step);
  }
  __device__ __forceinline__ void store(unsigned char *t, int tid) const {
    if (TL::NC < W && tid % W >= TL::NC) return;
#pragma unroll
    for (int i = 0; i < N; ++i)
      *reinterpret_cast<uint4 *>(t + TL::at(tid / W, tid % W) + i * R / 4 * TL::FOUR + i * R % 4 * TL::ROW) = r[i];
  }
};

// A chunk of an owned row straight from memory (zeros past head_dim or when
// the row is not there).
template <typename T, int DH>
__device__ __forceinline__ uint4 owned_chunk(const char *row, bool there, int chunk, int hd) {
  if (!there || chunk * Tile<T, DH>::E >= hd) return make_uint4(0, 0, 0, 0);
  return *reinterpret_cast<const uint4 *>(row + chunk * 16);
}

// Elements of a fragment replaced: `KEEP` its finite ones with zeros for the rest,
// `SIGN` the sign of its infinities and zeros for the rest, `ONE` ones for
// infinities and NaN and zeros for the rest.
enum class Part { KEEP, SIGN, ONE };
template <typename T, Part P>
__device__ __forceinline__ uint4 part_of(const uint4 &x) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      uint32_t r = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t v = w[i] >> (16 * k) & 0xffffu;
        const bool fin = (v & 0x7f80u) != 0x7f80u, inf = (v & 0x7fffu) == 0x7f80u;
        const uint32_t n = P == Part::KEEP ? (fin ? v : 0u)
                           : P == Part::SIGN ? (inf ? (v & 0x8000u) | 0x3f80u : 0u) : (fin ? 0u : 0x3f80u);
        r |= n << (16 * k);
      }
      w[i] = r;
    } else {
      const uint32_t v = w[i];
      const bool fin = (v & 0x7f800000u) != 0x7f800000u, inf = (v & 0x7fffffffu) == 0x7f800000u;
      w[i] = P == Part::KEEP ? (fin ? v : 0u)
             : P == Part::SIGN ? (inf ? (v & 0x80000000u) | 0x3f800000u : 0u) : (fin ? 0u : 0x3f800000u);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Asks the scheduler for a pipeline over the last N products: the LDS reads of AHEAD of
// them first, then a product and the reads (READS each) of a later one in turn.  Left
// alone it reads one fragment, waits for it and multiplies.
template <int N, int READS, int MFMAS, int AHEAD>
__device__ __forceinline__ void read_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, READS * AHEAD, 0);
#pragma unroll
  for (int i = 0; i < N - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, MFMAS, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, MFMAS * AHEAD, 0);
}

// Marks loaded fragments as arrived.  Without it the wait for them stands at their first
// use, inside the loop over tiles, where it waits for the next tile's loads as well.
template <int N>
__device__ __forceinline__ void arrived(uint4 (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(f[i].x), "+v"(f[i].y), "+v"(f[i].z), "+v"(f[i].w));
}

// The same for fragments that are to stay in accumulation registers, from which a product
// takes an operand as well as from a vector register.
template <int N>
__device__ __forceinline__ void arrived_acc(uint4 (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+a"(f[i].x), "+a"(f[i].y), "+a"(f[i].z), "+a"(f[i].w));
}

// Whether rows r0 .. r0+31 of a tile hold an infinity or a NaN (uniform): the
// largest bit pattern without its sign, two operations for a dword.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
template <typename T, int DH>
__device__ __forceinline__ bool not_finite(const unsigned char *t, int r0, int lane) {
  using TL = Tile<T, DH>;
  u16x2 top16 = {0, 0};
  uint32_t top32 = 0;
#pragma unroll
  for (int s = 0; s < TL::KS; ++s) {
    const uint4 x = TL::rows(t, r0, s, lane);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2)
        top16 = __builtin_elementwise_max(top16, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
      else
        top32 = max(top32, w[i] & 0x7fffffffu);
    }
  }
  const bool bad = sizeof(T) == 2 ? max(top16[0], top16[1]) >= 0x7f80u : top32 >= 0x7f800000u;
  return __ballot(bad) != 0;
}

// acc += tile^T p over rows r0 .. r0+31 of which some hold an infinity or a NaN:
// the product of the finite values, as ever and bit for bit, then what the
// others make of the sums of the owned rows that see them.  With S the sum
// of sign(value) sign(p) over seen infinities and Q the count of seen
// infinities and NaN, both products as well: nothing for Q = 0, +infinity for
// S = Q, -infinity for S = -Q, else NaN.
template <typename T, int DH>
__device__ __forceinline__ void sum_rows_guarded(const unsigned char *t, int r0, const f32x16 &p, uint32_t seen,
                                                 f32x16 (&acc)[DH / 32], int lane) {
  using TL = Tile<T, DH>;
  f32x16 one, sign;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    one[i] = seen >> i & 1u ? 1.f : 0.f;
    sign[i] = p[i] > 0.f ? one[i] : p[i] < 0.f ? -one[i] : 0.f;
  }
#pragma unroll
  for (int d = 0; d < TL::ND; ++d) {
    f32x16 sum, count;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[i] = count[i] = 0.f;
#pragma unroll
    for (int s = 0; s < TL::PS; ++s) {
      const uint4 x = TL::cols(t, r0, s, d, lane);
      mma_step<T>(part_of<T, Part::KEEP>(x), score_frag<T>(p, s), acc[d]);
      mma_step<T>(part_of<T, Part::SIGN>(x), score_frag<T>(sign, s), sum);
      mma_step<T>(part_of<T, Part::ONE>(x), score_frag<T>(one, s), count);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float with = acc[d][i] + (sum[i] == count[i] ? INFINITY : sum[i] == -count[i] ? -INFINITY : NAN);
      acc[d][i] = count[i] != 0.f ? with : acc[d][i];
    }
  }
}

// acc += tile^T p over rows r0 .. r0+31.
template <typename T, int DH>
__device__ __forceinline__ void sum_rows(const unsigned char *t, int r0, const f32x16 &p, f32x16 (&acc)[DH / 32],
                                         int lane) {
  using TL = Tile<T, DH>;
#pragma unroll
  for (int s = 0; s < TL::PS; ++s) {
    const uint4 b = score_frag<T>(p, s);
#pragma unroll
    for (int d = 0; d < TL::ND; ++d) mma_step<T>(TL::cols(t, r0, s, d, lane), b, acc[d]);
  }
}

// acc += tile^T of what p loses when it is rounded to bf16 (KEPT: of the tile's finite values),
// for short rows: where few keys and queries meet, few roundings are
// averaged.  bf16, 3 tokens, error of dq and dk against 64 bits over that of their own rounding: 1.4
// (1.7 at worst) without it, 1.0 with it; at 1000 tokens 1.4 (1.5) in any case without it.
template <bool KEPT, typename T, int DH>
__device__ __forceinline__ void sum_rows_rest(const unsigned char *t, int r0, const f32x16 &p, f32x16 (&acc)[DH / 32],
                                              int lane) {
  using TL = Tile<T, DH>;
  if constexpr (sizeof(T) == 2) {
    f32x16 rest;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = p[i] - (float)(bf16)p[i];
      rest[i] = x == x ? x : 0.f;  // (an infinite p)
    }
#pragma unroll
    for (int s = 0; s < TL::PS; ++s) {
      const uint4 b = score_frag<T>(rest, s);
#pragma unroll
      for (int d = 0; d < TL::ND; ++d) {
        const uint4 x = TL::cols(t, r0, s, d, lane);
        mma_step<T>(KEPT ? part_of<T, Part::KEEP>(x) : x, b, acc[d]);
      }
    }
  }
}

// In a tile where some row is not seen by some owned row, a product with that pair's zero p would
// carry an infinity or a NaN of the row to where it is not seen.  A kernel's first
// pass (GUARD false) only notes that it met one in such a tile; its block then starts
// over with GUARD, where such tiles take sum_rows_guarded.  (Both in one loop would keep the
// registers of the rare path from the common one.)
template <bool GUARD, typename T, int DH>
__device__ __forceinline__ void sum_rows_masked(const unsigned char *t, int r0, const f32x16 &p, uint32_t seen,
                                                f32x16 (&acc)[DH / 32], bool &met, int lane) {
  if constexpr (GUARD) {
    if (not_finite<T, DH>(t, r0, lane)) sum_rows_guarded<T, DH>(t, r0, p, seen, acc, lane);
    else sum_rows<T, DH>(t, r0, p, acc, lane);
  } else {
    met |= not_finite<T, DH>(t, r0, lane);
  }
}

// Writes 32 columns (from 32 d on) of an accumulator block times f into a row of T.
template <typename T>
__device__ __forceinline__ void write_part(char *row, const f32x16 &acc, int d, float f, int hd, int lane) {
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int col = 32 * d + 8 * b + 4 * (lane >> 5);
    if (col >= hd) continue;
    if constexpr (sizeof(T) == 2) {
      bf16 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (bf16)(acc[4 * b + i] * f);
      *reinterpret_cast<uint2 *>(row + col * 2) = __builtin_bit_cast(uint2, *(const u32x2 *)w);
    } else {
      *reinterpret_cast<float4 *>(row + col * 4) =
          make_float4(acc[4 * b] * f, acc[4 * b + 1] * f, acc[4 * b + 2] * f, acc[4 * b + 3] * f);
    }
  }
}
template <typename T, int DH>
__device__ __forceinline__ void write_row(char *row, const f32x16 (&acc)[DH / 32], float f, int hd, int lane) {
#pragma unroll
  for (int d = 0; d < DH / 32; ++d) write_part<T>(row, acc[d], d, f, hd, lane);
}

// Waves of the forward and dq kernels on a SIMD: as many as the registers of a wave allow (3 and not 2
// for bf16 heads of 64: 12 heads, 8 rows of 2048 tokens, forward 81 -> 75 us; 1 for rows of 512 bytes,
// whose owned rows alone take 128 registers).
template <typename T, int DH>
constexpr int waves() {
  return sizeof(T) * DH > 256 ? 1 : sizeof(T) * DH == 128 && sizeof(T) == 2 ? 3 : 2;
}

// With no more than one block of 128 queries for a CU the chip waits for the longest chain of
// keys.  The forward and dq then take blocks of 32 queries whose 4 waves share the keys, every
// fourth tile of 32 each in LDS of its own, and join their sums at the end: four times the
// blocks, a quarter of the chain.  bf16, forward, without and with: 12 heads of 64, 1024 tokens
// (96 blocks) 20 and 11 us; 8 of 128, 4096 (256) 87 and 74; 16 of 128, 4096 (512) 103 and 124;
// 16 rows of 128 tokens, 12 of 64 (192): 8.1 and 9.9, a chain too short to be worth a join.
constexpr int kFewBlocks = 256;
inline bool few_blocks(const AttnArgs &a) {
  const int64_t blocks = (int64_t)((a.T + 127) / 128) * a.H * a.B;
  return blocks <= kFewBlocks && blocks <= a.T / 2;
}

// Rows, or packed documents on average, short enough to take sum_rows_rest in their masked tiles, and
// in all of the few-block kernels' (whose tiles of 32 keys need no mask in rows of 33 tokens on; those of 64
// are masked in any document of up to 64).  Its products and registers cost 4096 rows of 16 tokens
// (12 heads of 64) 363 -> 385 us forward and 1262 -> 1432 backward, 8192 tokens in 256 documents 21 -> 25 us
// forward and 130 -> 149 forward and backward (16 + 4 heads of 128: 44 -> 48, 255 -> 286), one row of 37 nothing; they
// would cost packed rows of 16384 (heads of 128) 5 % of the forward, of 8192 15 % of forward and
// backward, where the sums average the roundings.
template <typename T>
inline bool with_rest(const AttnArgs &a) {
  return sizeof(T) == 2 && a.T <= 64 * (int64_t)(a.cu ? a.n_seqs : 1);
}

template <typename T, int DH>
struct FewLds {
  union {
    unsigned char tile[4][2][Tile<T, DH>::bytes(32)];  // [wave][key, value]
    float sum[4][DH / 2][64];                          // [wave][accumulator register][lane]
  };
  float top[4][32], tot[4][32];
};
// A wave's own LDS written before it is read (by other lanes).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Blocks over (tile, head, batch row): the tiles with most work first, and,
// where the heads divide among the 8 XCDs, a head's tiles on one XCD (block b
// runs on XCD b % 8), so that its keys and values stay in that XCD's L2.
__device__ __forceinline__ void block_of(int n_heads_all, int &tile_rank, int &head) {
  const int b = blockIdx.x;
  if (n_heads_all % 8 == 0) {
    const int per = n_heads_all / 8, i = b >> 3;
    head = (b & 7) * per + i % per;
    tile_rank = i / per;
  } else {
    head = b % n_heads_all;
    tile_rank = b / n_heads_all;
  }
}

int attn_fwd(const AttnArgs &a, int dtype, hipStream_t st);
int attn_bwd(const AttnArgs &a, int dtype, hipStream_t st);
int attn_bwd_fp32(const AttnArgs &a, hipStream_t st);
// blocks that share the (query head, query tile) pairs of a tile of keys in the dk/dv kernel
int attn_bwd_splits(const AttnArgs &a, int dtype);

}  // namespace dynconv
