// attn_paged.h -- arguments of the calls on a cache kept in pages (attn_paged.hip, attn_paged_store.hip).
#pragma once

#include "attn.h"
#include "pages.h"

namespace dynconv {

struct Pages {
  AttnView k, v;  // [n_pages, page_size, G, hd]: batch is the page's stride
  const int32_t *table;
  int64_t table_row;  // elements from one sequence's entries to the next one's
  int n_pages, size;
  int capacity;  // positions of a sequence's list
};

// Where row `slot` of a page starts in its pool.
__device__ __forceinline__ int64_t page_row(const AttnView &v, int page, int slot) {
  return (int64_t)page * v.batch + (int64_t)slot * v.row;
}

struct PagedArgs {
  AttnView q, k, v, o;
  Pages pages;
  int B, H, G, hd;
  int window, sinks;  // window 0: all cached tokens are seen
  int rot;            // 0: no rotation
  bool interleaved;
  float scale, factor;
  const double *freqs;
  const int32_t *lengths;
  int blocks;    // of the flat launch, 0: a block for each sequence and unit (key/value head and up to 16 query heads)
  int abreast;   // flat: units of a sequence that a block takes side by side
  float *part;   // flat: sums [2 blocks][abreast][columns][hd], then maximum and sum [2 blocks][abreast][columns][2]
  int2 *spans;   // flat: the first and the last block of each sequence and unit
};
int paged_abreast(const PagedArgs &a);
int paged_blocks(const PagedArgs &a);
int64_t paged_workspace(const PagedArgs &a);
int attn_paged(const PagedArgs &a, int dtype, hipStream_t st);

struct PagedStoreArgs {
  AttnView k, v;
  Pages pages;
  int B, T, G, hd;
  int rot;
  bool interleaved;
  float factor;
  const double *freqs;
  const int32_t *starts, *counts, *cu;  // any of them NULL
  int n_seqs;
};
// vec: bytes of an access that the pairs are made of (16, 8, or 0: single elements)
int attn_paged_store(const PagedStoreArgs &a, int dtype, int vec_bytes, hipStream_t st);

}  // namespace dynconv
