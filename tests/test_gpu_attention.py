"""Causal attention over whole sequences (dynconv_attn_fwd, dynconv_attn_bwd)
against its fp64 definition: head layouts, odd lengths and widths, packed
documents with empty and one-token ones and a padded end, views of one row and
head-major views, infinities and NaN where a row does not look, gradients
against differences, repeatability, replay in a HIP graph, two streams."""
from __future__ import annotations

import math
import sys

import pytest
import torch

import input_dependent_depthwise_amd as dc
from tests import attn_util as au

pytestmark = pytest.mark.gpu


def _note(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _row(B, T, H, G, hd, dtype, seed):
    """q, k, v as the parts of one row, and d_o."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = au.DTYPES[dtype]
    row = torch.randn(B, T, H + 2 * G, hd, generator=g, device="cuda").to(dt)
    d_o = torch.randn(B, T, H, hd, generator=g, device="cuda").to(dt)
    return row[:, :, :H], row[:, :, H:H + G], row[:, :, H + G:], d_o


def _run(q, k, v, d_o, cu=None, scale=None):
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, lse = dc.dynconv_attn_fwd(q, k, v, cu_seqlens=c, scale=scale, want_lse=True)
    g = dc.dynconv_attn_bwd(q, k, v, o, lse, d_o, cu_seqlens=c, scale=scale)
    torch.cuda.synchronize()
    return {"o": o, "lse": lse, **g}


def _compare(got, ref, dtype):
    # (2^-20: fp32 sums of up to 128 products, 2^-24 each)
    errs = {n: au.rel(got[n], ref[n], 2.0 ** -20 * ref.get("~" + n, 0.0)) for n in ref if n[0] != "~"}
    assert all(e <= (1e-5 if n == "lse" else au.TOL[dtype]) for n, e in errs.items()), errs


SHAPES = [
    # B, T, H, G, hd
    (1, 1, 1, 1, 64),
    (2, 1, 4, 2, 128),
    (1, 2, 3, 1, 16),
    (1, 31, 2, 2, 64),
    (2, 33, 4, 4, 16),
    (1, 64, 2, 1, 128),
    (3, 65, 6, 3, 80),
    (1, 127, 8, 1, 96),
    (1, 128, 8, 8, 8),
    (2, 129, 4, 2, 64),
    (1, 200, 7, 1, 128),
    (2, 257, 2, 1, 24),
    (1, 515, 12, 12, 64),
    (1, 1030, 16, 4, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_definition(shape, dtype):
    _note(f"[attn] {shape} {dtype}")
    q, k, v, d_o = _row(*shape, dtype, seed=sum(shape))
    _compare(_run(q, k, v, d_o), au.attention(q, k, v, d_o=d_o), dtype)


PACKED = [
    # offsets, T (the rest of the row is padding)
    ([0, 5], 5),
    ([0, 0, 1, 1, 2, 40, 40], 40),
    ([0, 31, 64, 65, 130], 130),
    ([0, 100, 228, 300], 333),
    ([0, 0, 0], 20),
    ([0, 7, 7, 128, 129, 512, 700], 700),
    ([0] + list(range(3, 600, 3)), 640),
    ([0, 126, 1000], 1027),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128), (3, 1, 40)], ids=str)
@pytest.mark.parametrize("docs", PACKED, ids=[f"docs{i}" for i in range(len(PACKED))])
def test_packed_documents(docs, heads, dtype):
    cu, T = docs
    H, G, hd = heads
    _note(f"[attn] packed {len(cu) - 1} documents T={T} {heads} {dtype}")
    q, k, v, d_o = _row(1, T, H, G, hd, dtype, seed=T + H)
    got = _run(q, k, v, d_o, cu=cu)
    _compare(got, au.attention(q, k, v, cu=cu, d_o=d_o), dtype)
    for n in ("o", "dq", "dk", "dv"):  # tokens of no document: exact zeros
        assert bool((got[n][:, cu[-1]:] == 0).all()), n
    assert bool((got["lse"][:, :, cu[-1]:] == -math.inf).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scale_and_large_scores(dtype):
    """Scores of some hundreds: the running maximum moves often and most probabilities vanish."""
    _note(f"[attn] large scores {dtype}")
    q, k, v, d_o = _row(2, 300, 4, 2, 64, dtype, seed=5)
    got, ref = _run(q, k, v, d_o, scale=6.0), au.attention(q, k, v, scale=6.0, d_o=d_o)
    # scores of |s| <= 300 carry an absolute error of |s| 2^-23 or so (fp32 sums), which p takes on as
    # a relative one, and near ties do.v - delta cancels
    for n in got:
        assert au.rel(got[n], ref[n]) <= (1e-5 if n == "lse" else au.TOL["bf16"] if dtype == "bf16" else 2e-4), n


def test_views():
    """Head-major tensors, heads shared by stride 0, gradients into the parts of one row: bitwise as for plain tensors."""
    _note("[attn] views")
    q, k, v, d_o = _row(2, 150, 4, 2, 64, "bf16", seed=9)
    ref = _run(q.contiguous(), k.contiguous(), v.contiguous(), d_o)
    hm = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731  [B, heads, T, head_dim] in memory
    got = _run(hm(q), hm(k), hm(v), hm(d_o))
    assert all(torch.equal(got[n], ref[n]) for n in ref)
    row = torch.full((2, 150, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = {"dq": row[:, :, :4], "dk": row[:, :, 4:6], "dv": row[:, :, 6:]}
    dc.dynconv_attn_bwd(q, k, v, ref["o"], ref["lse"], d_o, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], ref[n]) for n in out)
    one_k, one_v = k[:, :, :1].expand(-1, -1, 2, -1), v[:, :, :1].expand(-1, -1, 2, -1)
    got = _run(q, one_k, one_v, d_o)
    ref = _run(q, one_k.contiguous(), one_v.contiguous(), d_o)
    assert all(torch.equal(got[n], ref[n]) for n in ref)


BAD = [math.inf, -math.inf, math.nan, 3.0e38]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bad", BAD, ids=str)
def test_masked_places_do_not_reach(bad, hd, dtype):
    """One document, the padding and the later tokens of a row hold what would spoil a product with a zero."""
    _note(f"[attn] {bad} in masked places {hd} {dtype}")
    cu, T = [0, 40, 75, 170], 200
    q, k, v, d_o = _row(1, T, 4, 2, hd, dtype, seed=13)
    want = _run(q, k, v, d_o, cu=cu)
    q2, k2, v2, d2 = (t.clone() for t in (q, k, v, d_o))
    for t in (q2, k2, v2, d2):
        t[:, 40:75] = bad    # the second document
        t[:, 170:] = bad     # the padding
    got = _run(q2, k2, v2, d2, cu=cu)
    for n in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[n][:, :40], want[n][:, :40]), n
        assert torch.equal(got[n][:, 75:170], want[n][:, 75:170]), n
        assert bool((got[n][:, 170:] == 0).all()), n
    # later tokens: rows before them see nothing of it
    v3, k3 = v.clone(), k.clone()
    v3[:, 20:40] = bad
    k3[:, 20:40] = bad
    got = _run(q, k3, v3, d_o, cu=cu)
    assert torch.equal(got["o"][:, :20], want["o"][:, :20])
    assert torch.equal(got["dq"][:, :20], want["dq"][:, :20])


def test_gradients_against_differences():
    """Central differences of sum(o * d_o) along random directions (fp32 outputs, fp64 sums, step 1/64:
    truncation of order step^2, rounding 2^-24 / step)."""
    _note("[attn] differences")
    q, k, v, d_o = (t.contiguous() for t in _row(1, 90, 4, 2, 32, "fp32", seed=21))
    cu = [0, 33, 90]
    g = _run(q, k, v, d_o, cu=cu)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(22)
    step = 1 / 64
    for name, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        x = [q, k, v]
        d = torch.randn(x[i].shape, generator=gen, device="cuda")

        def loss(sign):
            y = list(x)
            y[i] = x[i] + sign * step * d
            return (dc.dynconv_attn_fwd(*y, cu_seqlens=c).double() * d_o.double()).sum()

        num = ((loss(1) - loss(-1)) / (2 * step)).item()
        ana = (g[name].double() * d.double()).sum().item()
        size = g[name].double().norm().item() * math.sqrt(d.numel()) / math.sqrt(g[name].numel()) + 1.0
        assert abs(num - ana) <= 1e-2 * size, (name, num, ana, size)


def test_repeatable_and_on_two_streams():
    _note("[attn] repeat, two streams")
    q, k, v, d_o = _row(2, 700, 8, 2, 128, "bf16", seed=31)
    ref = _run(q, k, v, d_o)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        out = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                o, lse = dc.dynconv_attn_fwd(q, k, v, want_lse=True)
                out.append({"o": o, "lse": lse, **dc.dynconv_attn_bwd(q, k, v, o, lse, d_o)})
        torch.cuda.synchronize()
        for got in out:
            assert all(torch.equal(got[n], ref[n]) for n in ref)


def test_graph_replay():
    _note("[attn] graph")
    q, k, v, d_o = (t.contiguous() for t in _row(1, 333, 4, 2, 64, "bf16", seed=41))
    c = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")

    def step():
        o, lse = dc.dynconv_attn_fwd(q, k, v, cu_seqlens=c, want_lse=True)
        return {"o": o, "lse": lse, **dc.dynconv_attn_bwd(q, k, v, o, lse, d_o, cu_seqlens=c)}

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(3):
        for t, n in zip((q, k, v, d_o), _row(1, 333, 4, 2, 64, "bf16", seed=50 + r)):
            t.copy_(n)
        c.copy_(torch.tensor([0, 60 + r, 333 - r], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], eager[n]) for n in eager), r


def test_empty():
    q = torch.empty(0, 5, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert dc.dynconv_attn_fwd(q, q, q).shape == q.shape
    q = torch.empty(2, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = dc.dynconv_attn_fwd(q, q, q, want_lse=True)
    g = dc.dynconv_attn_bwd(q, q, q, o, lse, q)
    torch.cuda.synchronize()
    assert lse.shape == (2, 4, 0) and g["dk"].shape == q.shape


# Enough blocks of 128 queries for the chip (the shapes above have fewer and take blocks of 32).
LARGE = [
    (16, 260, 8, 2, 128),
    (32, 130, 12, 12, 64),
    (22, 129, 6, 3, 16),
    (13, 385, 7, 1, 96),
    (2, 2100, 8, 4, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_many_blocks_against_definition(shape, dtype):
    _note(f"[attn] {shape} {dtype}")
    q, k, v, d_o = _row(*shape, dtype, seed=sum(shape))
    _compare(_run(q, k, v, d_o), au.attention(q, k, v, d_o=d_o), dtype)


LONG_ROW = [0, 0, 1, 40, 171, 171, 300, 1500, 1564, 1628, 1700, 4100]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (9, 3, 64), (12, 12, 24)], ids=str)
def test_many_blocks_packed(heads, dtype):
    H, G, hd = heads
    _note(f"[attn] long packed row {heads} {dtype}")
    q, k, v, d_o = _row(1, 4200, H, G, hd, dtype, seed=H)
    got = _run(q, k, v, d_o, cu=LONG_ROW)
    _compare(got, au.attention(q, k, v, cu=LONG_ROW, d_o=d_o), dtype)
    for n in ("o", "dq", "dk", "dv"):
        assert bool((got[n][:, 4100:] == 0).all()), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bad", BAD, ids=str)
def test_many_blocks_masked_places(bad, hd, dtype):
    _note(f"[attn] {bad} in masked places of a long row {hd} {dtype}")
    cu = [0, 700, 760, 2500, 4100]
    q, k, v, d_o = _row(1, 4200, 8, 4, hd, dtype, seed=17)
    want = _run(q, k, v, d_o, cu=cu)
    q2, k2, v2, d2 = (t.clone() for t in (q, k, v, d_o))
    for t in (q2, k2, v2, d2):
        t[:, 700:760] = bad
        t[:, 4100:] = bad
    got = _run(q2, k2, v2, d2, cu=cu)
    for n in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[n][:, :700], want[n][:, :700]), n
        assert torch.equal(got[n][:, 760:4100], want[n][:, 760:4100]), n
        assert bool((got[n][:, 4100:] == 0).all()), n
    v3 = v.clone()
    v3[:, 1000:1100] = bad
    got = _run(q, k, v3, d_o, cu=cu)
    assert torch.equal(got["o"][:, :1000], want["o"][:, :1000])


def test_seen_infinities():
    """What a row does see of them it keeps: +infinity, -infinity or NaN as in the sum itself."""
    _note("[attn] seen infinities")
    for T, H in ((200, 2), (4200, 8)):
        q, k, v, _ = _row(1, T, H, H, 64, "fp32", seed=19)
        v[:, 50, :, 0], v[:, 60, :, 0], v[:, 70, :, 1], v[:, 80, :, 2] = math.inf, -math.inf, math.nan, -math.inf
        ref = au.attention(q, k, v)["o"]
        got = dc.dynconv_attn_fwd(q, k, v)
        assert au.rel(got, ref) <= au.TOL["fp32"]
        assert bool(torch.isinf(got[:, 50:60, :, 0]).all()) and bool(torch.isnan(got[:, 60:, :, 0]).all())
        assert bool(torch.isfinite(got[:, :50]).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", [(6, 2, 96), (3, 3, 72), (4, 1, 88), (2, 1, 104)], ids=str)
@pytest.mark.parametrize("docs", [PACKED[3], PACKED[5], (LONG_ROW, 4200)], ids=["300", "700", "4100"])
def test_packed_heads_between_64_and_128(docs, heads, dtype):
    cu, T = docs
    H, G, hd = heads
    if T > 1000:  # enough blocks of 128
        H, G = 9 * G, 3 * G
    _note(f"[attn] packed {len(cu) - 1} documents T={T} {H} {G} {hd} {dtype}")
    q, k, v, d_o = _row(1, T, H, G, hd, dtype, seed=T + hd)
    got = _run(q, k, v, d_o, cu=cu)
    _compare(got, au.attention(q, k, v, cu=cu, d_o=d_o), dtype)
    for n in ("o", "dq", "dk", "dv"):
        assert bool((got[n][:, cu[-1]:] == 0).all()), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [333, 4200])
@pytest.mark.parametrize("bad", BAD, ids=str)
def test_masked_places_heads_of_96(bad, T, dtype):
    _note(f"[attn] {bad} in masked places, heads of 96, {T} tokens {dtype}")
    a, b, c = T // 6, T // 6 + 40, T - T // 40
    q, k, v, d_o = _row(1, T, 9, 3, 96, dtype, seed=T)
    want = _run(q, k, v, d_o, cu=[0, a, b, c])
    q2, k2, v2, d2 = (t.clone() for t in (q, k, v, d_o))
    for t in (q2, k2, v2, d2):
        t[:, a:b] = bad
        t[:, c:] = bad
    got = _run(q2, k2, v2, d2, cu=[0, a, b, c])
    for n in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[n][:, :a], want[n][:, :a]), n
        assert torch.equal(got[n][:, b:c], want[n][:, b:c]), n
        assert bool((got[n][:, c:] == 0).all()), n


@pytest.mark.parametrize("hd", [64, 96, 128])
@pytest.mark.parametrize("B,T", [(1, 2), (1, 3), (40, 5), (1, 31), (30, 32)])
def test_short_rows_in_bf16_lose_no_more_than_their_own_rounding(B, T, hd):
    """p and ds enter the products with 16 bits there (2^-17 each, against 2^-9 of the outputs' rounding)."""
    _note(f"[attn] own rounding {B} {T} {hd}")
    q, k, v, d_o = _row(B, T, 4, 2, hd, "bf16", seed=B + T + hd)
    got, ref = _run(q, k, v, d_o), au.attention(q, k, v, d_o=d_o)
    for n in ("o", "dq", "dk", "dv"):
        off = (got[n].double() - ref[n]).norm()
        own = (ref[n].bfloat16().double() - ref[n]).norm()
        assert off <= 1.1 * own + 2.0 ** -16 * ref[n].norm(), (n, float(off / own))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [24, 64, 80, 128])
@pytest.mark.parametrize("cu,T", [([0, 130, 100], 130), ([0, 40, 700, 90, 300], 520)], ids=["130", "520"])
def test_offsets_that_fall_stay_inside_the_row(cu, T, hd, dtype):
    """Offsets that break the rule give unspecified values, from the row's own tokens and into them alone."""
    _note(f"[attn] falling offsets {cu} T={T} {hd} {dtype}")
    H, G, room = 4, 2, 200
    q, k, v, d_o = _row(1, T, H, G, hd, dtype, seed=T + hd)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    seen = []
    for around in (0.0, 5.0):
        wide = [torch.full((1, T + 2 * room, t.shape[2], hd), around, dtype=t.dtype, device="cuda") for t in (q, k, v, d_o)]
        for w, t in zip(wide, (q, k, v, d_o)):
            w[:, room:room + T] = t
        x = [w[:, room:room + T] for w in wide]
        out = [torch.full_like(w, 7.0) for w in (wide[0], *wide[:3])]
        o, dq, dk, dv = (w[:, room:room + T] for w in out)
        _, lse = dc.dynconv_attn_fwd(*x[:3], cu_seqlens=c, o=o, want_lse=True)
        dc.dynconv_attn_bwd(*x[:3], o, lse, x[3], cu_seqlens=c, out={"dq": dq, "dk": dk, "dv": dv})
        torch.cuda.synchronize()
        for w in out:
            assert bool((w[:, :room] == 7).all()) and bool((w[:, room + T:] == 7).all())
        seen.append([t.clone() for t in (o, lse, dq, dk, dv)])
    assert all(torch.equal(a, b) for a, b in zip(*seen))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_smallest_scale(dtype):
    """At the smallest factor that a call takes all scores vanish: dv is the mean of do over the queries' keys."""
    _note(f"[attn] smallest scale {dtype}")
    q, k, v, d_o = _row(2, 300, 4, 2, 64, dtype, seed=23)
    _compare(_run(q, k, v, d_o, scale=2.0 ** -120), au.attention(q, k, v, scale=2.0 ** -120, d_o=d_o), dtype)
    for scale in (2.0 ** -121, 2.0 ** -126):
        with pytest.raises(ValueError):
            _run(q, k, v, d_o, scale=scale)


def _off_over_own(got, ref, rows):
    """The error over that of the definition rounded to bf16, both over the given [B, T] rows."""
    got, ref = got.double()[rows], ref[rows]
    return ((got - ref).norm() / (ref.bfloat16().double() - ref).norm()).item()


@pytest.mark.parametrize("H,G,hd", [(8, 2, 64), (8, 2, 128), (9, 3, 96)])
def test_few_keys_where_a_document_starts_before_a_block(H, G, hd):
    """Rows of 2 to 8 keys at the head of a block of 128 queries, their document starting just before it.  Two
    independent roundings to bf16 lie on the way to dq (ds and dq itself): 1.41 times dq's own; the rounding of o
    in delta would make it 2.3."""
    _note(f"[attn] documents across blocks {H} {G} {hd}")
    T = 128 * 40
    cu = [0] + [128 * m - 1 - m % 7 for m in range(1, 40)] + [T]
    q, k, v, d_o = _row(1, T, H, G, hd, "bf16", seed=H + hd)
    got, ref = _run(q, k, v, d_o, cu=cu), au.attention(q, k, v, cu=cu, d_o=d_o)
    t, start = torch.arange(T, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    for lo in cu[:-1]:
        start[lo:] = lo
    rows = ((t - start < 8) & (t - start > 0) & (t // 128 > start // 128))[None]
    assert int(rows.sum()) > 100
    assert _off_over_own(got["dq"], ref["dq"], rows) <= 1.7


@pytest.mark.parametrize("hd", [64, 96, 128])
@pytest.mark.parametrize("B,T", [(1, 33), (1, 60), (30, 60), (1, 64), (40, 64)])
def test_rows_of_up_to_64_tokens_in_bf16_lose_no_more_than_their_own_rounding(B, T, hd):
    """As above, with tiles that no mask cuts (keys 0 to 31 of queries 32 to 63)."""
    _note(f"[attn] own rounding {B} {T} {hd}")
    q, k, v, d_o = _row(B, T, 8, 4, hd, "bf16", seed=B + T + hd)
    got, ref = _run(q, k, v, d_o), au.attention(q, k, v, d_o=d_o)
    for n in ("o", "dq", "dk", "dv"):
        off = (got[n].double() - ref[n]).norm()
        own = (ref[n].bfloat16().double() - ref[n]).norm()
        assert off <= 1.1 * own + 2.0 ** -16 * ref[n].norm(), (n, float(off / own))


@pytest.mark.parametrize("hd", [64, 96, 128])
@pytest.mark.parametrize("T,each,H", [(300, 3, 4), (600, 2, 4), (3900, 3, 9), (3910, 17, 9), (3968, 64, 9)])
def test_packed_short_documents_in_bf16_lose_no_more_than_their_own_rounding(T, each, H, hd):
    """The same documents as in rows of their own, behind one another in one row."""
    _note(f"[attn] own rounding of documents of {each} in {T} {hd}")
    cu = list(range(0, T + 1, each))
    q, k, v, d_o = _row(1, T, H, H // 2 if H % 2 == 0 else 3, hd, "bf16", seed=T + hd)
    got, ref = _run(q, k, v, d_o, cu=cu), au.attention(q, k, v, cu=cu, d_o=d_o)
    for n in ("o", "dq", "dk", "dv"):
        off = (got[n].double() - ref[n]).norm()
        own = (ref[n].bfloat16().double() - ref[n]).norm()
        assert off <= 1.1 * own + 2.0 ** -16 * ref[n].norm(), (n, float(off / own))


def test_gradients_into_parts_of_one_buffer():
    """dq, dk and dv side by side in one buffer on any axis, tokens outside the batch or a group's heads together:
    bitwise as in tensors of their own."""
    _note("[attn] parts of one buffer")
    B, T, H, G, hd = 2, 150, 4, 2, 64
    q, k, v, d_o = _row(B, T, H, G, hd, "bf16", seed=29)
    o, lse = dc.dynconv_attn_fwd(q, k, v, want_lse=True)
    want = dc.dynconv_attn_bwd(q, k, v, o, lse, d_o)
    new = lambda *shape: torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    tokens_outside = new(T, B, H + 2 * G, hd).transpose(0, 1)
    head_major = new(B, H + 2 * G, T, hd).transpose(1, 2)
    for row in (tokens_outside, head_major):
        out = {"dq": row[:, :, :H], "dk": row[:, :, H:H + G], "dv": row[:, :, H + G:]}
        dc.dynconv_attn_bwd(q, k, v, o, lse, d_o, out=out)
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in want)
    groups = new(B, T, G, 3, hd)
    one = q[:, :, :G]
    o, lse = dc.dynconv_attn_fwd(one, k, v, want_lse=True)
    want = dc.dynconv_attn_bwd(one, k, v, o, lse, d_o[:, :, :G])
    out = {n: groups[:, :, :, i] for i, n in enumerate(("dq", "dk", "dv"))}
    dc.dynconv_attn_bwd(one, k, v, o, lse, d_o[:, :, :G], out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in want)


@pytest.mark.parametrize("B,T,H,G,hd", [(2, 129, 4, 2, 64), (1, 515, 12, 12, 64), (1, 1030, 16, 4, 128), (2, 257, 4, 1, 80),
                                        (16, 260, 8, 2, 128), (2, 2100, 8, 4, 64)])
def test_longer_rows_in_bf16_add_one_rounding_to_their_own(B, T, H, G, hd):
    """p or ds rounded once and the output rounded once, independent of each other and of like size: 1.41 times
    the output's own.  A product that lost one more bit would be at 2.2."""
    _note(f"[attn] one rounding more {B} {T} {H} {G} {hd}")
    q, k, v, d_o = _row(B, T, H, G, hd, "bf16", seed=T + hd)
    got, ref = _run(q, k, v, d_o), au.attention(q, k, v, d_o=d_o)
    every = torch.ones(B, T, dtype=torch.bool, device="cuda")
    errs = {n: _off_over_own(got[n], ref[n], every) for n in ("o", "dq", "dk", "dv")}
    assert all(e <= 1.75 for e in errs.values()), errs
