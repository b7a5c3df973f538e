"""The row ranges that the attention kernels take from packed documents' offsets
(csrc/docs.h), compiled for the host: the definition's for offsets that keep the
rule, and within the row's tokens for any others (device data the host cannot check)."""
from __future__ import annotations

import os
import subprocess

import input_dependent_depthwise_amd as dc

CSRC = os.path.join(os.path.dirname(dc.__file__), "csrc")

PROGRAM = r"""
#define __host__
#define __device__
#define __forceinline__ inline
#include <stdio.h>
#include <stdlib.h>
#include "docs.h"
using namespace dynconv;

static int fail(const char *what, const int32_t *cu, int n, int T, int at) {
  printf("%s T=%d at=%d cu=[", what, T, at);
  for (int i = 0; i <= n; ++i) printf(" %d", cu[i]);
  printf(" ]\n");
  return 1;
}

// A tile of `rows` rows from row0 on, read up to `limit`: every byte that a lane can reach lies
// in the T rows (row_bytes apart, len bytes each); lanes past the head ask for `outside`.
static bool inside(int row0, int limit, int T, int64_t row_bytes, int len) {
  const uint32_t outside = 0x80000000u;
  const uint32_t size = rows_extent(row0, limit, row_bytes, len, outside);
  return row0 >= 0 && size <= outside && (size == 0 || row0 * row_bytes + (int64_t)size <= (T - 1) * row_bytes + len);
}

static int check(const int32_t *cu, int n, int T, bool good) {
  const int limit = tokens_in_docs(cu, n, T);
  if (limit < 0 || limit > T) return fail("limit", cu, n, T, limit);
  for (int t = 0; t < T; ++t) {
    int start, end;
    doc_of(cu, n, T, limit, t, start, end);
    if (end > limit || start < 0 || (start > t && start != T)) return fail("document", cu, n, T, t);
    if (!good) continue;
    int s = T, e = 0;
    for (int i = 0; i < n; ++i)
      if (cu[i] <= t && t < cu[i + 1]) s = cu[i], e = cu[i + 1];
    if (start != s || end != e) return fail("wrong document", cu, n, T, t);
  }
  for (int rows = 32; rows <= 128; rows += 96)
    for (int r0 = 0; r0 < T; r0 += rows) {
      int first, last;
      keys_of(cu, n, T, limit, r0, rows, first, last);
      if (first < 0 || last >= limit) return fail("keys", cu, n, T, r0);
      for (int kt = first; kt <= last; kt += 32)
        if (kt >= limit || !inside(kt, limit, T, 256, 160)) return fail("key tile", cu, n, T, r0);
      const int stop = queries_end(cu, n, T, limit, r0, rows);
      if (stop > limit) return fail("queries", cu, n, T, r0);
      for (int qt = r0; qt < stop; qt += 32)
        if (qt >= limit || !inside(qt, limit, T, 256, 160)) return fail("query tile", cu, n, T, r0);
      if (good) {
        int s = T, e = 0;
        for (int i = 0; i < n; ++i)
          for (int t = r0; t < r0 + rows && t < T; ++t)
            if (cu[i] <= t && t < cu[i + 1]) s = cu[i] < s ? cu[i] : s, e = cu[i + 1] > e ? cu[i + 1] : e;
        if (first <= last && first != s) return fail("first key", cu, n, T, r0);
        if (stop > r0 ? stop != e : e != 0) return fail("last query", cu, n, T, r0);
      }
    }
  return 0;
}

int main() {
  // the last offset below an earlier one: the document that ends at 130 ends at 100
  const int32_t falls[] = {0, 130, 100};
  if (check(falls, 2, 130, false)) return 1;
  if (rows_extent(128, 100, 256, 160, 0x80000000u) != 0) return fail("extent", falls, 2, 130, 128);
  if (check(NULL, 0, 300, false)) return 1;
  srand(5);
  for (int r = 0; r < 20000; ++r) {
    int32_t cu[9];
    const int n = 1 + rand() % 8, T = 1 + rand() % 400;
    const bool good = r % 2;
    for (int i = 0; i <= n; ++i)
      cu[i] = rand() % 16 ? rand() % (T + 1) : good ? 0 : rand() % 2 ? -rand() % 500 : 2147483647 - rand() % 300;
    if (good) {
      cu[0] = 0;
      for (int i = 1; i <= n; ++i)
        for (int j = i; j > 0 && cu[j] < cu[j - 1]; --j) { const int32_t x = cu[j]; cu[j] = cu[j - 1]; cu[j - 1] = x; }
    }
    if (check(cu, n, T, good)) return 1;
  }
  printf("ok\n");
  return 0;
}
"""


def test_ranges(tmp_path):
    src, exe = tmp_path / "docs.cpp", tmp_path / "docs"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unused-function", "-Wno-unused-variable", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
