// attn_api.hip -- C entry points of the Q/K/V path behind the convolution
// (rotary positions, attention, its backward, the decode step): validation on
// the host, then kernel dispatch.  Declared in include/dynconv.h.
#include <math.h>

#include <algorithm>

#include "attn_decode.h"
#include "kernels.h"
#include "rope.h"

namespace dynconv {

namespace {

constexpr int64_t kMaxRow = 16 << 20;  // bytes between tokens: 64 rows stay below 2 GiB

// The bf16 dk/dv kernel starts its sums at -lse / scale: the logarithm of up to 2^31 keys over this
// is below 2^125 (at 2^-126 rows of 55 keys and more passed the largest float, and their p came out as 0).
constexpr float kLeastScale = 0x1p-120f;

struct Extent {  // what a view covers, in bytes
  const char *p;
  int64_t batch, row, head;  // strides, 0 for axes of length 1
  int64_t B, T, H, len;      // len: bytes of one head
  int64_t span;              // from p to past the last element
};

// A non-negative stride in elements as bytes, 0 where the axis has one entry
// (the stride then means nothing).  Refuses what would pass 2^62 bytes in all.
int stride_bytes(int64_t n, int64_t stride, int64_t eb, bool vectors, int64_t &out) {
  out = 0;
  if (n <= 1) return DYNCONV_OK;
  if (stride < 0) return DYNCONV_E_SHAPE;
  if (stride > ((int64_t)1 << 60) / n / eb) return DYNCONV_E_LIMIT;
  out = stride * eb;
  return vectors && out % 16 != 0 ? DYNCONV_E_ALIGN : DYNCONV_OK;
}

// vectors: the kernel reads and writes whole 16-byte vectors.
int extent(const dynconv_view *v, int64_t B, int64_t T, int64_t H, int64_t hd, int64_t eb, bool vectors, Extent &x) {
  if (!v || !v->data) return DYNCONV_E_NULL;
  int rc;
  if ((rc = stride_bytes(B, v->batch, eb, vectors, x.batch)) || (rc = stride_bytes(T, v->row, eb, vectors, x.row)) ||
      (rc = stride_bytes(H, v->head, eb, vectors, x.head)))
    return rc;
  if ((uintptr_t)v->data % (vectors ? 16 : eb) != 0) return DYNCONV_E_ALIGN;
  if (vectors && x.row > kMaxRow) return DYNCONV_E_LIMIT;
  x.p = (const char *)v->data;
  x.B = B;
  x.T = T;
  x.H = H;
  x.len = hd * eb;
  x.span = (B - 1) * x.batch + (T - 1) * x.row + (H - 1) * x.head + x.len;
  return DYNCONV_OK;
}

// No element of an output twice: each axis strides past what the shorter strides cover.
bool disjoint_rows(const Extent &x) {
  int64_t s[3] = {x.batch, x.row, x.head}, n[3] = {x.B, x.T, x.H};
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int i, int j) { return s[i] < s[j]; });
  int64_t cover = x.len;
  for (int i : order) {
    if (n[i] <= 1) continue;
    if (s[i] < cover) return false;
    cover = s[i] * (n[i] - 1) + cover;
  }
  return true;
}

// Whether two views might share an element.  Views that interleave in one buffer (heads of one row, rows of
// one batch, on whatever axis they alternate) are told apart by a stride of one of them as a period: strides that
// are multiples of it do not matter then, and what the others cover of each view has to lie beside the
// other's within the period.
bool meet(const Extent &a, const Extent &b) {
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  if (a0 + (uint64_t)a.span <= b0 || b0 + (uint64_t)b.span <= a0) return false;
  const int64_t d = (int64_t)(b0 - a0);
  auto cover = [](const Extent &x, int64_t period) {  // bytes from its first element on, modulo the period
    const int64_t s[3] = {x.batch, x.row, x.head}, n[3] = {x.B, x.T, x.H};
    int64_t c = x.len;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && s[i] % period != 0) c += (n[i] - 1) * s[i];
    return c;
  };
  for (int64_t period : {a.batch, a.row, a.head, b.batch, b.row, b.head}) {
    if (period <= 0) continue;
    const int64_t ca = cover(a, period), cb = cover(b, period), m = ((d % period) + period) % period;
    if (m >= ca && m + cb <= period) return false;
  }
  return true;
}

Extent flat(const void *p, int64_t bytes) { return {(const char *)p, 0, 0, 0, 1, 1, 1, bytes, bytes}; }

AttnView strided(const Extent &x) { return {const_cast<char *>(x.p), x.batch, x.row, x.head}; }

// Sizes shared by the calls.  attention: head layout, scale and block counts as well.
int check_attn(const dynconv_attn *a, bool attention) {
  if (!a) return DYNCONV_E_NULL;
  if (a->dtype != DYNCONV_FP32 && a->dtype != DYNCONV_BF16) return DYNCONV_E_DTYPE;
  if (a->B < 0 || a->T < 0 || a->n_heads <= 0 || a->head_dim <= 0) return DYNCONV_E_SHAPE;
  const int64_t lim = ((int64_t)1 << 31) - 4096;
  if (a->B > lim || a->T > lim || a->n_heads > 65535) return DYNCONV_E_LIMIT;
  if (attention) {
    if (a->n_kv_heads <= 0 || a->n_heads % a->n_kv_heads != 0) return DYNCONV_E_SHAPE;
    if (a->head_dim % (a->dtype == DYNCONV_BF16 ? 8 : 4) != 0) return DYNCONV_E_SHAPE;
    if (!(a->scale == 0.f || a->scale >= kLeastScale) || isinf(a->scale)) return DYNCONV_E_SHAPE;
    if (a->head_dim > 128) return DYNCONV_E_LIMIT;
    // blocks of 256 threads, below 2^32 threads in all
    if (a->B > 0 && a->T > 0 && (a->T + 127) / 128 > (((int64_t)1 << 24) - 1) / a->n_heads / a->B) return DYNCONV_E_LIMIT;
  }
  if (a->cu_seqlens) {
    if (a->B != 1 || a->n_seqs < 1) return DYNCONV_E_SHAPE;
    if (((uintptr_t)a->cu_seqlens & 3u) != 0) return DYNCONV_E_ALIGN;
    if (a->n_seqs >= lim) return DYNCONV_E_LIMIT;
  }
  return DYNCONV_OK;
}

int check_rotary(const dynconv_rotary *r, int head_dim) {
  if (!r || !r->freqs) return DYNCONV_E_NULL;
  if (r->rot_dim <= 0 || r->rot_dim % 2 != 0 || r->rot_dim > head_dim) return DYNCONV_E_SHAPE;
  if (((uintptr_t)r->freqs & 7u) != 0) return DYNCONV_E_ALIGN;
  return DYNCONV_OK;
}

float scale_of(const dynconv_attn *a) {
  return a->scale > 0.f ? a->scale : (float)(1.0 / sqrt((double)a->head_dim));
}

AttnArgs attn_args(const dynconv_attn *a) {
  AttnArgs r = {};
  r.B = (int)a->B;
  r.T = (int)a->T;
  r.H = a->n_heads;
  r.G = a->n_kv_heads;
  r.hd = a->head_dim;
  r.n_split = 1;
  r.scale = scale_of(a);
  r.cu = a->cu_seqlens;
  r.n_seqs = a->cu_seqlens ? (int)a->n_seqs : 0;
  return r;
}

inline int attn_status() { return hipGetLastError() == hipSuccess ? DYNCONV_OK : DYNCONV_E_HIP; }
inline int64_t pad256(int64_t v) { return (v + 255) / 256 * 256; }

// Backward workspace: delta, then the partial dk / dv.
struct BwdPlan {
  int splits;
  int64_t delta, part;
};
BwdPlan bwd_plan(const dynconv_attn *a) {
  BwdPlan p;
  p.splits = attn_bwd_splits(attn_args(a), a->dtype);
  p.delta = pad256(a->B * a->n_heads * a->T * 4);
  p.part = p.splits > 1 ? (int64_t)2 * p.splits * a->B * a->n_kv_heads * a->T * a->head_dim * 4 : 0;
  return p;
}

int64_t decode_bytes(const dynconv_attn *a, int64_t capacity) {
  const int n = decode_splits(a->B, a->n_heads, a->n_kv_heads, capacity);
  return n > 1 ? a->B * a->n_heads * n * (a->head_dim + 2) * 4 : 0;
}

}  // namespace

}  // namespace dynconv

using namespace dynconv;

extern "C" {

int dynconv_rope_freqs(int rot_dim, double base, double stretch, double trained_len, double slow_turns,
                       double fast_turns, double *out) {
  if (!out) return DYNCONV_E_NULL;
  if (rot_dim <= 0 || rot_dim % 2 != 0 || !(base > 0.0) || !(stretch >= 1.0) || !(trained_len >= 0.0) ||
      isinf(base) || isinf(stretch) || isinf(trained_len) || (trained_len > 0.0 && !(fast_turns > slow_turns)))
    return DYNCONV_E_SHAPE;
  for (int m = 0; m < rot_dim / 2; ++m) {
    const double f = pow(base, -2.0 * m / rot_dim);
    double keep = 0.0;
    if (trained_len > 0.0) {
      const double turns = trained_len * f / 6.283185307179586477;
      keep = fmin(fmax((turns - slow_turns) / (fast_turns - slow_turns), 0.0), 1.0);
    }
    out[m] = f * keep + f / stretch * (1.0 - keep);
  }
  return DYNCONV_OK;
}

int dynconv_rope(const dynconv_attn *a, const dynconv_rotary *r, const dynconv_view *x, const int32_t *positions,
                 const dynconv_view *y, hipStream_t stream) {
  int rc = check_attn(a, false);
  if (rc || (rc = check_rotary(r, a->head_dim))) return rc;
  if (a->B == 0 || a->T == 0) return DYNCONV_OK;
  const int64_t eb = a->dtype == DYNCONV_BF16 ? 2 : 4;
  Extent ex, ey;
  if ((rc = extent(x, a->B, a->T, a->n_heads, a->head_dim, eb, false, ex)) ||
      (rc = extent(y, a->B, a->T, a->n_heads, a->head_dim, eb, false, ey)))
    return rc;
  if (positions && ((uintptr_t)positions & 3u) != 0) return DYNCONV_E_ALIGN;
  const int64_t lim = ((int64_t)1 << 31) - 4096;
  if (a->B > lim / a->T || a->B * a->T > lim * 256 / a->head_dim) return DYNCONV_E_LIMIT;
  // the kernels count the vectors of a token and the bytes of a head in 32 bits
  if (a->n_heads > lim / (a->head_dim * eb)) return DYNCONV_E_LIMIT;
  const bool in_place = ex.p == ey.p && ex.batch == ey.batch && ex.row == ey.row && ex.head == ey.head;
  if (!disjoint_rows(ey) || (!in_place && meet(ex, ey))) return DYNCONV_E_ALIAS;
  const Extent others[] = {flat(r->freqs, r->rot_dim / 2 * 8), flat(positions, positions ? a->B * a->T * 4 : 0),
                           flat(a->cu_seqlens, a->cu_seqlens ? (a->n_seqs + 1) * 4 : 0)};
  for (const Extent &o : others)
    if (o.p && meet(ey, o)) return DYNCONV_E_ALIAS;
  // the widest vector that both views, their strides and the halves of the pairs are made of
  int vec = 0;
  for (int64_t w : {8, 16}) {
    const int64_t all = (int64_t)(uintptr_t)ex.p | (int64_t)(uintptr_t)ey.p | ex.batch | ex.row | ex.head | ey.batch |
                        ey.row | ey.head | a->head_dim * eb | r->rot_dim / 2 * eb;
    if (all % w == 0 && w / eb >= 2) vec = (int)w;
  }
  RopeArgs k = {ex.p,
                const_cast<char *>(ey.p),
                ex.batch,
                ex.row,
                ex.head,
                ey.batch,
                ey.row,
                ey.head,
                (int)a->B,
                (int)a->T,
                a->n_heads,
                a->head_dim,
                r->rot_dim,
                r->interleaved != 0,
                in_place,
                r->factor,
                r->inverse ? -1.f : 1.f,
                r->freqs,
                positions,
                a->cu_seqlens,
                a->cu_seqlens ? (int)a->n_seqs : 0};
  if ((rc = rope(k, a->dtype, vec, stream))) return rc;
  return attn_status();
}

int dynconv_attn_fwd(const dynconv_attn *a, const dynconv_view *q, const dynconv_view *k, const dynconv_view *v,
                     const dynconv_view *o, float *lse, hipStream_t stream) {
  int rc = check_attn(a, true);
  if (rc) return rc;
  if (a->B == 0 || a->T == 0) return DYNCONV_OK;
  const int64_t eb = a->dtype == DYNCONV_BF16 ? 2 : 4, H = a->n_heads, G = a->n_kv_heads, hd = a->head_dim;
  Extent xq, xk, xv, xo;
  if ((rc = extent(q, a->B, a->T, H, hd, eb, true, xq)) || (rc = extent(k, a->B, a->T, G, hd, eb, true, xk)) ||
      (rc = extent(v, a->B, a->T, G, hd, eb, true, xv)) || (rc = extent(o, a->B, a->T, H, hd, eb, true, xo)))
    return rc;
  if (lse && ((uintptr_t)lse & 3u) != 0) return DYNCONV_E_ALIGN;
  const Extent xl = flat(lse, lse ? a->B * H * a->T * 4 : 0);
  const Extent xc = flat(a->cu_seqlens, a->cu_seqlens ? (a->n_seqs + 1) * 4 : 0);
  if (!disjoint_rows(xo)) return DYNCONV_E_ALIAS;
  const Extent *ins[] = {&xq, &xk, &xv, &xc};
  for (const Extent *i : ins) {
    if (!i->p) continue;
    if (meet(xo, *i) || (lse && meet(xl, *i))) return DYNCONV_E_ALIAS;
  }
  if (lse && meet(xo, xl)) return DYNCONV_E_ALIAS;
  AttnArgs r = attn_args(a);
  r.q = strided(xq);
  r.k = strided(xk);
  r.v = strided(xv);
  r.o = strided(xo);
  r.lse = lse;
  if ((rc = attn_fwd(r, a->dtype, stream))) return rc;
  return attn_status();
}

size_t dynconv_attn_bwd_workspace_bytes(const dynconv_attn *a) {
  if (check_attn(a, true) || a->B == 0 || a->T == 0) return 0;
  const BwdPlan p = bwd_plan(a);
  return (size_t)(p.delta + p.part);
}

int dynconv_attn_bwd(const dynconv_attn *a, const dynconv_view *q, const dynconv_view *k, const dynconv_view *v,
                     const dynconv_view *o, const float *lse, const dynconv_view *d_o, const dynconv_view *dq,
                     const dynconv_view *dk, const dynconv_view *dv, void *workspace, size_t workspace_bytes,
                     hipStream_t stream) {
  int rc = check_attn(a, true);
  if (rc) return rc;
  if (a->B == 0 || a->T == 0) return DYNCONV_OK;
  const int64_t eb = a->dtype == DYNCONV_BF16 ? 2 : 4, H = a->n_heads, G = a->n_kv_heads, hd = a->head_dim;
  if (!lse) return DYNCONV_E_NULL;
  const dynconv_view *views[] = {q, k, v, o, d_o, dq, dk, dv};
  const int64_t heads[] = {H, G, G, H, H, H, G, G};
  Extent x[8];
  for (int i = 0; i < 8; ++i)
    if ((rc = extent(views[i], a->B, a->T, heads[i], hd, eb, true, x[i]))) return rc;
  if (((uintptr_t)lse & 3u) != 0 || ((uintptr_t)workspace & 15u) != 0) return DYNCONV_E_ALIGN;
  const BwdPlan p = bwd_plan(a);
  if (!workspace || workspace_bytes < (size_t)(p.delta + p.part)) return DYNCONV_E_WORKSPACE;
  const Extent xl = flat(lse, a->B * H * a->T * 4);
  const Extent xc = flat(a->cu_seqlens, a->cu_seqlens ? (a->n_seqs + 1) * 4 : 0);
  const Extent xw = flat(workspace, p.delta + p.part);
  const Extent *ins[] = {&x[0], &x[1], &x[2], &x[3], &x[4], &xl, &xc}, *outs[] = {&x[5], &x[6], &x[7], &xw};
  for (int i = 0; i < 4; ++i) {
    if (i < 3 && !disjoint_rows(*outs[i])) return DYNCONV_E_ALIAS;
    for (const Extent *n : ins)
      if (n->p && meet(*outs[i], *n)) return DYNCONV_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (meet(*outs[i], *outs[j])) return DYNCONV_E_ALIAS;
  }
  AttnArgs r = attn_args(a);
  r.q = strided(x[0]);
  r.k = strided(x[1]);
  r.v = strided(x[2]);
  r.o = strided(x[3]);
  r.d_o = strided(x[4]);
  r.dq = strided(x[5]);
  r.dk = strided(x[6]);
  r.dv = strided(x[7]);
  r.lse = const_cast<float *>(lse);
  r.delta = (float *)workspace;
  r.part = (float *)((char *)workspace + p.delta);
  r.n_split = p.splits;
  if ((rc = attn_bwd(r, a->dtype, stream))) return rc;
  return attn_status();
}

size_t dynconv_attn_decode_workspace_bytes(const dynconv_attn *a, int64_t capacity) {
  if (check_attn(a, true) || a->B == 0 || capacity <= 0) return 0;
  return (size_t)decode_bytes(a, capacity);
}

int dynconv_attn_decode(const dynconv_attn *a, const dynconv_rotary *rot, const dynconv_view *q,
                        const dynconv_view *k, const dynconv_view *v, const dynconv_view *k_cache,
                        const dynconv_view *v_cache, int64_t capacity, const int32_t *lengths, const dynconv_view *o,
                        void *workspace, size_t workspace_bytes, hipStream_t stream) {
  int rc = check_attn(a, true);
  if (rc) return rc;
  if (a->T != 1 || a->cu_seqlens || capacity <= 0) return DYNCONV_E_SHAPE;
  if (capacity > ((int64_t)1 << 31) - 4096 || a->B > 65535 || a->n_kv_heads * ((a->n_heads / a->n_kv_heads + 15) / 16) > 65535)
    return DYNCONV_E_LIMIT;
  if (rot && (rc = check_rotary(rot, a->head_dim))) return rc;
  if (rot && rot->inverse) return DYNCONV_E_SHAPE;
  if (a->B == 0) return DYNCONV_OK;
  const int64_t eb = a->dtype == DYNCONV_BF16 ? 2 : 4, H = a->n_heads, G = a->n_kv_heads, hd = a->head_dim;
  if (!lengths) return DYNCONV_E_NULL;
  Extent xq, xk, xv, xo, xkc, xvc;
  if ((rc = extent(q, a->B, 1, H, hd, eb, true, xq)) || (rc = extent(k, a->B, 1, G, hd, eb, true, xk)) ||
      (rc = extent(v, a->B, 1, G, hd, eb, true, xv)) || (rc = extent(o, a->B, 1, H, hd, eb, true, xo)) ||
      (rc = extent(k_cache, a->B, capacity, G, hd, eb, true, xkc)) ||
      (rc = extent(v_cache, a->B, capacity, G, hd, eb, true, xvc)))
    return rc;
  if (((uintptr_t)lengths & 3u) != 0 || ((uintptr_t)workspace & 15u) != 0) return DYNCONV_E_ALIGN;
  const int64_t need = decode_bytes(a, capacity);
  if (need > 0 && (!workspace || workspace_bytes < (size_t)need)) return DYNCONV_E_WORKSPACE;
  const Extent xw = flat(need > 0 ? workspace : nullptr, need);
  const Extent xn = flat(lengths, a->B * 4), xf = flat(rot ? rot->freqs : nullptr, rot ? rot->rot_dim / 2 * 8 : 0);
  const Extent *ins[] = {&xq, &xk, &xv, &xn, &xf}, *outs[] = {&xo, &xkc, &xvc, &xw};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]->p) continue;
    if (i < 3 && !disjoint_rows(*outs[i])) return DYNCONV_E_ALIAS;
    for (const Extent *n : ins)
      if (n->p && meet(*outs[i], *n)) return DYNCONV_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (meet(*outs[i], *outs[j])) return DYNCONV_E_ALIAS;
  }
  DecodeArgs r = {};
  r.q = strided(xq);
  r.k = strided(xk);
  r.v = strided(xv);
  r.o = strided(xo);
  r.kc = strided(xkc);
  r.vc = strided(xvc);
  r.B = (int)a->B;
  r.H = a->n_heads;
  r.G = a->n_kv_heads;
  r.hd = a->head_dim;
  r.capacity = (int)capacity;
  r.n_split = decode_splits(a->B, a->n_heads, a->n_kv_heads, capacity);
  r.rot = rot ? rot->rot_dim : 0;
  r.interleaved = rot && rot->interleaved != 0;
  r.scale = scale_of(a);
  r.factor = rot ? rot->factor : 1.f;
  r.freqs = rot ? rot->freqs : nullptr;
  r.lengths = lengths;
  r.part = (float *)workspace;
  if ((rc = attn_decode(r, a->dtype, stream))) return rc;
  return attn_status();
}

}  // extern "C"
