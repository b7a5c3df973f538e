// docs.h -- packed documents: which rows the attention kernels' tiles take.
// Plain integer arithmetic, usable on the host as well.  The offsets are device
// data that nobody has checked: whatever they hold, every range here lies within
// the row's tokens [0, T), and a tile starts below the limit it is read up to.
#pragma once

#include <stdint.h>

namespace dynconv {

__host__ __device__ __forceinline__ int lesser(int a, int b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int greater(int a, int b) { return a > b ? a : b; }

// Tokens of the row that belong to a document (all T without packing).
__host__ __device__ __forceinline__ int tokens_in_docs(const int32_t *cu, int n_seqs, int T) {
  if (!cu) return T;
  return lesser(greater(cu[n_seqs], 0), T);
}

// The document of token t: [start, end), 0 <= start <= t and end <= limit
// (limit: tokens_in_docs).  A token of none gets start = T and end = 0.
__host__ __device__ __forceinline__ void doc_of(const int32_t *cu, int n_seqs, int T, int limit, int t, int &start,
                                                int &end) {
  if (!cu) {
    start = t < T ? 0 : T;
    end = t < T ? T : 0;
    return;
  }
  int lo = 0, hi = n_seqs;  // the first j in [1, n_seqs] with cu[j] > t, else n_seqs + 1
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  if (lo >= n_seqs || t >= limit) {
    start = T;
    end = 0;
    return;
  }
  start = lesser(greater(cu[lo], 0), t);
  end = lesser(cu[lo + 1], limit);
}

// The keys that queries q0 .. q0 + rows - 1 see: first .. last, none when first > last.
__host__ __device__ __forceinline__ void keys_of(const int32_t *cu, int n_seqs, int T, int limit, int q0, int rows,
                                                 int &first, int &last) {
  int unused;
  doc_of(cu, n_seqs, T, limit, q0, first, unused);
  last = lesser(q0 + rows - 1, limit - 1);
}

// The queries that see keys k0 .. k0 + rows - 1: from k0 up to this one, none when it is not above k0.
__host__ __device__ __forceinline__ int queries_end(const int32_t *cu, int n_seqs, int T, int limit, int k0, int rows) {
  if (k0 >= limit) return 0;
  int unused, end;
  doc_of(cu, n_seqs, T, limit, lesser(k0 + rows - 1, limit - 1), unused, end);
  return end;
}

// Bytes that a read of rows row0 .. limit - 1 (row_bytes apart, `len` bytes each) may reach from row0 on, at
// most `most`; nothing when there is no such row.
__host__ __device__ __forceinline__ uint32_t rows_extent(int row0, int limit, int64_t row_bytes, int len, uint32_t most) {
  if (row0 >= limit) return 0;
  const int64_t bytes = (int64_t)(limit - row0 - 1) * row_bytes + len;
  return bytes < (int64_t)most ? (uint32_t)bytes : most;
}

}  // namespace dynconv
