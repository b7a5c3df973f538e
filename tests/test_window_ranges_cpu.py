"""The ranges that the windowed attention kernels take (csrc/docs.h), compiled for the host: every key that some
query of a block sees lies in exactly one of its tiles, every query that sees a key in its block's near or
far part, and each sum of the far part is written in the slot where it is read."""
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
#include <set>
#include <tuple>
#include <vector>
#include "docs.h"
using namespace dynconv;

static int fail(const char *what, const int32_t *cu, int n, int T, int W, int S, int at) {
  printf("%s T=%d window=%d sinks=%d at=%d cu=[", what, T, W, S, at);
  for (int i = 0; cu && i <= n; ++i) printf(" %d", cu[i]);
  printf(" ]\n");
  return 1;
}

static int check(const int32_t *cu, int n, int T, int W, int S, bool good, int kFarChunk) {
  const int kFarSlots = kFarChunk / 128;
  const int limit = tokens_in_docs(cu, n, T);
  std::vector<int> start(T), end(T);
  for (int t = 0; t < T; ++t) doc_of(cu, n, T, limit, t, start[t], end[t]);
  auto sees = [&](int q, int k) {
    return end[q] > 0 && k <= q && k >= start[q] && (q - k < W || k < start[q] + S);
  };
  for (int rows = 32; rows <= 128; rows += 96)
    for (int tile = 32; tile <= 64; tile += 32)
      for (int q0 = 0; q0 < T; q0 += rows) {
        int first, last, hop_at, hop_to;
        keys_of(cu, n, T, limit, q0, rows, first, last);
        window_keys(W, S, tile, q0, first, hop_at, hop_to);
        std::vector<char> in(T, 0);
        int count = 0;
        for (int kt = first; kt <= last; kt = kt + tile == hop_at ? hop_to : kt + tile) {
          if (kt < 0 || kt >= limit || ++count > T) return fail("tile", cu, n, T, W, S, q0);
          for (int k = kt; k < kt + tile && k < T; ++k) ++in[k];
        }
        // the same by index
        for (int i = 0, kt = first; i < count; ++i, kt = kt + tile == hop_at ? hop_to : kt + tile) {
          const int x = first + tile * i;
          if ((hop_at < 0 || x < hop_at ? x : hop_to + (x - hop_at)) != kt) return fail("index", cu, n, T, W, S, q0);
        }
        if (!good) continue;
        for (int q = q0; q < q0 + rows && q < T; ++q)
          for (int k = 0; k <= q; ++k)
            if (sees(q, k) && in[k] != 1) return fail(in[k] ? "key twice" : "key lost", cu, n, T, W, S, q);
        if (count > (W + rows + tile - 2) / tile + (S + tile - 1) / tile + 1) return fail("tiles", cu, n, T, W, S, q0);
      }
  // near and far queries of each key
  std::set<std::tuple<int, int, int>> wrote, read;  // chunk, slot, sink's key
  std::vector<std::vector<char>> seen(T, std::vector<char>(T, 0));
  for (int k0 = 0; k0 < T; k0 += 128) {
    const int doc_end = queries_end(cu, n, T, limit, k0, 128), stop = window_end(W, k0, 128, doc_end);
    if (stop > limit) return fail("stop", cu, n, T, W, S, k0);
    for (int k = k0; k < k0 + 128 && k < T; ++k) {
      int e = end[k];
      if (k >= start[k] + S) e = window_end(W, k, 1, e);
      e = lesser(e, stop);
      for (int q = k; q < e; ++q) ++seen[k][q];
    }
    if (k0 < limit && stop < doc_end && S > 0) {
      const int st = start[lesser(k0 + 127, limit - 1)];
      for (int s = greater(k0, st); s < lesser(k0 + 128, st + S); ++s)
        for (int c = stop / kFarChunk; c <= (doc_end - 1) / kFarChunk; ++c) {
          const int slot = cu ? far_slot(kFarChunk, c, st) : 0;
          if (slot < 0 || slot >= (cu ? kFarSlots : 1) || s - st < 0 || s - st >= S || c * kFarChunk >= T)
            return fail("read outside", cu, n, T, W, S, s);
          read.insert({c, slot, s});
        }
    }
  }
  for (int c = 0; c * kFarChunk < T; ++c)
    for (int m = 0, done = -1; m < (cu ? kFarSlots : 1) && S > 0; ++m) {
      const int t = c * kFarChunk + (m ? 128 * m - 1 : 0);
      int st, en;
      doc_of(cu, n, T, limit, t, st, en);
      if (en == 0 || st == done) continue;
      done = st;
      const int slot = cu ? far_slot(kFarChunk, c, st) : 0;
      for (int s = st, k; s < lesser(st + S, en); s += k) {
        const int k0 = s / 128 * 128;
        k = lesser(lesser(st + S, k0 + 128) - s, 32);
        const int from = greater(c * kFarChunk, window_end(W, k0, 128, en)), to = lesser((c + 1) * kFarChunk, en);
        if (from >= to) continue;
        if (slot < 0 || slot >= (cu ? kFarSlots : 1) || k <= 0 || to > limit) return fail("write outside", cu, n, T, W, S, s);
        for (int x = s; x < s + k; ++x) {
          if (good && !wrote.insert({c, slot, x}).second) return fail("slot twice", cu, n, T, W, S, x);
          for (int q = from; q < to; ++q) ++seen[x][q];
        }
      }
    }
  if (!good) return 0;
  for (auto &r : read)
    if (!wrote.count(r)) return fail("slot not written", cu, n, T, W, S, std::get<2>(r));
  if (read.size() != wrote.size()) return fail("slot not read", cu, n, T, W, S, 0);
  for (int k = 0; k < T; ++k)
    for (int q = 0; q < T; ++q)
      if (seen[k][q] != (char)sees(q, k)) return fail(seen[k][q] > 1 ? "pair twice" : "pair", cu, n, T, W, S, q);
  return 0;
}

int main() {
  srand(7);
  for (int r = 0; r < 700; ++r) {
    int32_t cu[9];
    const int n = 1 + rand() % 8, T = 1 + rand() % (r % 7 ? 700 : 2300);
    const int W = rand() % 3 ? 1 + rand() % 150 : 1 + rand() % T, S = rand() % 4 ? rand() % 20 : rand() % 129;
    const bool good = r % 4 != 0;
    for (int i = 0; i <= n; ++i)
      cu[i] = rand() % 16 ? rand() % (T + 1) : good ? 0 : rand() % 2 ? -rand() % 500 : 2147483647 - rand() % 300;
    if (good) {
      cu[0] = 0;
      for (int i = 1; i <= n; ++i)
        for (int j = i; j > 0 && cu[j] < cu[j - 1]; --j) { const int32_t x = cu[j]; cu[j] = cu[j - 1]; cu[j - 1] = x; }
    }
    if (check(r % 5 ? cu : NULL, n, T, W, S, r % 5 ? good : true, 128 << r % 4)) return 1;
  }
  printf("ok\n");
  return 0;
}
"""


def test_ranges(tmp_path):
    src, exe = tmp_path / "ranges.cpp", tmp_path / "ranges"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wno-unused-function", "-Wno-unused-variable", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
