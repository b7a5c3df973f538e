// pages.h -- which tokens of a cache kept in pages the kernels read and store.  Plain integer arithmetic, usable on
// the host as well.  Lengths, starts, offsets and tables are device data that nobody has checked: whatever they hold, a position
// taken from here lies in [0, capacity) and a page in [0, n_pages).
#pragma once

#include "docs.h"

namespace dynconv {

constexpr int kGroup = 32;  // cached tokens a wave takes at a time

// The groups of a sequence with n cached tokens, 0 <= n < capacity: group 0 is the new token at position n, the others
// are of the cache, those with sinks before the window and those from the window's first token on.
struct Seen {
  int n;       // cached tokens
  int from;    // those from here on are in the window
  int sinks;   // and those before this one are sinks
  int ns, g0;  // groups of sinks before the window's groups, the first of which is g0
  int groups;  // with the new token's
};
__host__ __device__ __forceinline__ Seen seen_of(int window, int sinks, int n) {  // window 0: none
  Seen s;
  s.n = n;
  s.from = window ? greater(0, n + 1 - window) : 0;
  s.sinks = lesser(sinks, s.from);
  s.g0 = s.from / kGroup;
  s.ns = lesser((s.sinks + kGroup - 1) / kGroup, s.g0);
  s.groups = 1 + s.ns + greater(0, (n + kGroup - 1) / kGroup - s.g0);
  return s;
}
// The first token of a group from 1 on.
__host__ __device__ __forceinline__ int first_key(const Seen &s, int group) {
  const int i = group - 1;
  return (i < s.ns ? i : s.g0 + i - s.ns) * kGroup;
}
__host__ __device__ __forceinline__ bool sees(const Seen &s, int key) {
  return key < s.n && (key >= s.from || key < s.sinks);
}

// Sequence and position of a token of k [B, T] that is to be stored, -1 for one that is not.
__host__ __device__ __forceinline__ int stored_at(const int32_t *cu, int n_seqs, const int32_t *starts,
                                                  const int32_t *counts, int T, int capacity, int64_t token, int &seq) {
  int64_t t;
  seq = 0;
  if (cu) {
    const int limit = tokens_in_docs(cu, n_seqs, T);
    int lo = 0, hi = n_seqs;  // the first j in [1, n_seqs] with cu[j] > token, else n_seqs + 1
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid + 1] > token) hi = mid;
      else lo = mid + 1;
    }
    if (lo >= n_seqs || token >= limit) return -1;
    seq = lo;
    t = token - cu[lo];
  } else {
    seq = (int)(token / T);
    t = token - (int64_t)seq * T;
    if (counts && t >= counts[seq]) return -1;
  }
  const int start = starts ? starts[seq] : 0;
  const int64_t pos = start + t;
  return start < 0 || t < 0 || pos >= capacity ? -1 : (int)pos;
}

// The page of a position of [0, capacity) in a sequence's list, -1 for none.
__host__ __device__ __forceinline__ int page_at(const int32_t *list, int size, int n_pages, int pos) {
  const int page = list[(uint32_t)pos / (uint32_t)size];
  return (uint32_t)page < (uint32_t)n_pages ? page : -1;
}

}  // namespace dynconv
