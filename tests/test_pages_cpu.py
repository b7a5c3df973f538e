"""The positions and pages that the calls on a cache kept in pages take (csrc/pages.h), compiled for the host: each
seen token in one group, each token of a prompt at its position, and nothing outside the lists and the pool whatever
lengths, starts, offsets and tables hold."""
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
#include <vector>
#include "pages.h"
using namespace dynconv;

static int check_seen(int window, int sinks, int n, int capacity) {
  const Seen s = seen_of(window, sinks, n);
  std::vector<int> count(capacity, 0);
  for (int g = 1; g < s.groups; ++g)
    for (int i = 0; i < kGroup; ++i) {
      const int key = first_key(s, g) + i;
      if (key < 0 || !sees(s, key)) continue;
      if (key >= capacity) { printf("outside %d %d %d %d\n", window, sinks, n, key); return 1; }
      ++count[key];
    }
  for (int j = 0; j < capacity; ++j) {
    const bool want = j < n && (!window || n - j < window || j < sinks);
    if (count[j] != (int)want) { printf("key %d %d times: %d %d %d\n", j, count[j], window, sinks, n); return 1; }
  }
  const int64_t reach = window ? (int64_t)window + sinks + 2 * kGroup : capacity;
  const int64_t most = 1 + ((reach < capacity ? reach : capacity) + kGroup - 1) / kGroup;
  if (s.groups < 1 || s.groups > most) { printf("groups %d of %d: %d %d %d\n", s.groups, (int)most, window, sinks, n); return 1; }
  return 0;
}

int main() {
  srand(3);
  for (int r = 0; r < 20000; ++r) {
    const int capacity = 1 + rand() % 600, n = rand() % capacity;
    const int window = rand() % 3 ? 1 + rand() % capacity : rand() % 2 ? 0 : 2147483647 - rand() % 3, sinks = window ? rand() % 129 : 0;
    if (check_seen(window, sinks, n, capacity)) return 1;
  }
  // far ends of what the numbers hold
  const int far = 2147483647 - 4097;
  for (int window : {0, 1, 31, 2147483647}) {
    const Seen s = seen_of(window, 128, far);
    const int64_t end = (int64_t)first_key(s, s.groups - 1) + kGroup;
    if (s.groups > 1 && (first_key(s, s.groups - 1) < 0 || end < far)) { printf("far %d\n", window); return 1; }
  }
  for (int r = 0; r < 20000; ++r) {
    int32_t cu[9], starts[8], counts[8], list[40];
    const int n = 1 + rand() % 8, T = 1 + rand() % 60, capacity = 1 + rand() % 100;
    const bool good = r % 2, packed = rand() % 2, has_starts = rand() % 4, has_counts = !packed && rand() % 2;
    auto wild = [&](int most) { return rand() % 3 ? rand() % most : rand() % 2 ? -2147483647 - 1 + rand() % 1000 : 2147483647 - rand() % 1000; };
    for (int i = 0; i <= n; ++i) cu[i] = good ? rand() % (T + 1) : wild(T + 1);
    for (int i = 0; i < n; ++i) starts[i] = good ? rand() % 30 - 2 : wild(30), counts[i] = good ? rand() % (T + 3) : wild(T);
    if (good) {
      cu[0] = 0;
      for (int i = 1; i <= n; ++i)
        for (int j = i; j > 0 && cu[j] < cu[j - 1]; --j) { const int32_t x = cu[j]; cu[j] = cu[j - 1]; cu[j - 1] = x; }
    }
    for (int64_t token = 0; token < (packed ? T : (int64_t)n * T); ++token) {
      int seq;
      const int pos = stored_at(packed ? cu : NULL, packed ? n : 0, has_starts ? starts : NULL, has_counts ? counts : NULL, T, capacity, token, seq);
      if (seq < 0 || (seq >= n && pos >= 0) || pos < -1 || pos >= capacity) { printf("position %d of %d\n", pos, seq); return 1; }
      if (!good) continue;
      int want = -1, b = (int)(token / T), t = (int)(token % T);
      if (packed) {
        b = -1;
        for (int i = 0; i < n; ++i)
          if (cu[i] <= token && token < cu[i + 1]) b = i, t = (int)token - cu[i];
      }
      const int s = b < 0 ? -1 : has_starts ? starts[b] : 0;
      if (s >= 0 && (!has_counts || t < counts[b]) && s + t < capacity) want = s + t;
      if (pos != want || (pos >= 0 && seq != b)) { printf("token %d: %d, not %d\n", (int)token, pos, want); return 1; }
    }
    const int size = 1 + rand() % 20, per = 1 + rand() % 40, n_pages = 1 + rand() % 50;
    for (int i = 0; i < per; ++i) list[i] = wild(60);
    for (int pos = 0; pos < size * per; ++pos) {
      const int page = page_at(list, size, n_pages, pos), e = list[pos / size];
      if (page != (e >= 0 && e < n_pages ? e : -1)) { printf("page %d of %d\n", page, e); return 1; }
    }
  }
  printf("ok\n");
  return 0;
}
"""


def test_positions(tmp_path):
    src, exe = tmp_path / "pages.cpp", tmp_path / "pages"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unused-function", "-Wno-unused-variable", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-2000:]
