"""Causal attention through a sliding window with sinks (dynconv_attn_window_fwd, dynconv_attn_window_bwd) against its
fp64 definition: windows from one token to the row, sinks before, across and inside it, head layouts, odd lengths
and widths, packed documents, views, infinities and NaN where a row does not look, gradients against
differences, repeatability, replay in a HIP graph, two streams."""
from __future__ import annotations

import math
import sys

import pytest
import torch

import input_dependent_depthwise_amd as dc
from tests import attn_util as au
from tests import window_util as wu

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


def _run(q, k, v, d_o, window, sinks=0, cu=None, scale=None):
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, lse = dc.dynconv_attn_window_fwd(q, k, v, window, sinks=sinks, cu_seqlens=c, scale=scale, want_lse=True)
    torch.cuda.synchronize()
    _note("  forward done")
    g = dc.dynconv_attn_window_bwd(q, k, v, o, lse, d_o, window, sinks=sinks, cu_seqlens=c, scale=scale)
    torch.cuda.synchronize()
    return {"o": o, "lse": lse, **g}


def _compare(got, ref, dtype):
    # (2^-20: fp32 sums of up to 128 products, 2^-24 each)
    errs = {n: au.rel(got[n], ref[n], 2.0 ** -20 * ref.get("~" + n, 0.0)) for n in ref if n[0] != "~"}
    assert all(e <= (1e-5 if n == "lse" else au.TOL[dtype]) for n, e in errs.items()), errs


CASES = [
    # (B, T, H, G, hd), window, sinks
    ((1, 1, 1, 1, 64), 1, 0),
    ((2, 2, 4, 2, 128), 1, 1),
    ((1, 31, 2, 2, 64), 7, 2),
    ((2, 33, 4, 4, 16), 1, 0),        # every token sees itself alone
    ((1, 37, 12, 12, 64), 16, 2),
    ((1, 64, 2, 1, 128), 63, 3),
    ((3, 65, 6, 3, 80), 20, 128),     # more sinks than tokens
    ((1, 129, 8, 1, 96), 64, 1),
    ((2, 200, 4, 2, 64), 100, 33),
    ((1, 300, 7, 1, 128), 1, 1),
    ((1, 515, 12, 12, 64), 129, 4),
    ((1, 700, 4, 2, 8), 40, 128),
    ((2, 1030, 8, 4, 128), 200, 4),
    ((1, 1030, 3, 1, 40), 1029, 4),
    ((1, 2100, 4, 1, 64), 65, 17),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[0])) + f"-{c[1]}-{c[2]}")
def test_against_definition(case, dtype):
    shape, window, sinks = case
    _note(f"[window] {shape} window {window} sinks {sinks} {dtype}")
    q, k, v, d_o = _row(*shape, dtype, seed=sum(shape) + window)
    _compare(_run(q, k, v, d_o, window, sinks), wu.attention(q, k, v, window, sinks, d_o=d_o), dtype)


# Enough blocks of 128 queries for the chip (the shapes above have fewer and take blocks of 32).
MANY = [
    ((16, 260, 8, 2, 128), 70, 3),
    ((32, 130, 12, 12, 64), 5, 1),
    ((22, 129, 6, 3, 16), 128, 0),
    ((13, 385, 7, 1, 96), 130, 40),
    ((2, 2100, 8, 4, 64), 300, 4),
    ((2, 2100, 8, 4, 128), 64, 128),
    ((1, 4200, 9, 3, 80), 1000, 5),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "x".join(map(str, c[0])) + f"-{c[1]}-{c[2]}")
def test_many_blocks_against_definition(case, dtype):
    shape, window, sinks = case
    _note(f"[window] {shape} window {window} sinks {sinks} {dtype}")
    q, k, v, d_o = _row(*shape, dtype, seed=sum(shape) + window)
    _compare(_run(q, k, v, d_o, window, sinks), wu.attention(q, k, v, window, sinks, d_o=d_o), dtype)


PACKED = [
    # offsets, T (the rest of the row is padding)
    ([0, 5], 5),
    ([0, 0, 1, 1, 2, 40, 40], 40),
    ([0, 100, 228, 300], 333),
    ([0, 0, 0], 20),
    ([0, 7, 7, 128, 129, 512, 700], 700),
    ([0] + list(range(3, 600, 3)), 640),
    ([0, 126, 1000], 1027),
    ([0, 60, 1300, 1301, 2300], 2310),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128), (3, 1, 40)], ids=str)
@pytest.mark.parametrize("window,sinks", [(1, 2), (30, 4), (150, 128)])
@pytest.mark.parametrize("docs", PACKED, ids=[f"docs{i}" for i in range(len(PACKED))])
def test_packed_documents(docs, window, sinks, heads, dtype):
    cu, T = docs
    H, G, hd = heads
    _note(f"[window] packed {len(cu) - 1} documents T={T} window {window} sinks {sinks} {heads} {dtype}")
    q, k, v, d_o = _row(1, T, H, G, hd, dtype, seed=T + H)
    got = _run(q, k, v, d_o, window, sinks, cu=cu)
    _compare(got, wu.attention(q, k, v, window, sinks, cu=cu, d_o=d_o), dtype)
    for n in ("o", "dq", "dk", "dv"):  # tokens of no document: exact zeros
        assert bool((got[n][:, cu[-1]:] == 0).all()), n
    assert bool((got["lse"][:, :, cu[-1]:] == -math.inf).all())


LONG_ROW = [0, 0, 1, 40, 171, 171, 300, 1500, 1564, 1628, 1700, 4100]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (9, 3, 64), (9, 3, 96), (12, 12, 24)], ids=str)
@pytest.mark.parametrize("window,sinks", [(50, 4), (513, 100)])
def test_many_blocks_packed(heads, window, sinks, dtype):
    H, G, hd = heads
    _note(f"[window] long packed row {heads} window {window} sinks {sinks} {dtype}")
    q, k, v, d_o = _row(1, 4200, H, G, hd, dtype, seed=H)
    got = _run(q, k, v, d_o, window, sinks, cu=LONG_ROW)
    _compare(got, wu.attention(q, k, v, window, sinks, cu=LONG_ROW, d_o=d_o), dtype)
    for n in ("o", "dq", "dk", "dv"):
        assert bool((got[n][:, 4100:] == 0).all()), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cu", [None, [0, 1000, 2100], [0, 37, 130, 2000, 2090]])
@pytest.mark.parametrize("heads", [(2, 1, 64), (8, 2, 128), (3, 3, 80)], ids=str)
@pytest.mark.parametrize("window,sinks", [(3, 128), (200, 33), (90, 7)])
def test_sinks_of_many_chunks(window, sinks, heads, cu, dtype):
    """Few heads over a long row: sinks 32 at a time in blocks of their own, chunks of several blocks' queries, shared among
    the splits of the sinks' tile, and added eight and four at a time."""
    _note(f"[window] many chunks {heads} window {window} sinks {sinks} docs {cu} {dtype}")
    q, k, v, d_o = _row(1, 2100, *heads, dtype, seed=window)
    _compare(_run(q, k, v, d_o, window, sinks, cu=cu), wu.attention(q, k, v, window, sinks, cu=cu, d_o=d_o), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_past_4_gib(dtype):
    """Rows a MiB apart: the last ones lie past 4 GiB from their tensor's start.  Bit for bit the call on dense tensors."""
    _note(f"[window] rows a MiB apart {dtype}")
    T, H, G, hd, window, sinks = 4500, 4, 2, 64, 70, 5
    q, k, v, d_o = _row(1, T, H, G, hd, dtype, seed=8)
    want = _run(q, k, v, d_o, window, sinks)
    wide = torch.zeros(1, T, 2 ** 20 // q.element_size(), dtype=q.dtype, device="cuda")
    at = 0

    def place(x):
        nonlocal at
        n = x.shape[2] * hd
        view = wide[:, :, at:at + n].view(1, T, x.shape[2], hd)
        at += n
        return view

    ins = [place(x) for x in (q, k, v, d_o)]
    for view, x in zip(ins, (q, k, v, d_o)):
        view.copy_(x)
    o = place(q)
    o, lse = dc.dynconv_attn_window_fwd(*ins[:3], window, sinks=sinks, o=o, want_lse=True)
    out = {"dq": place(q), "dk": place(k), "dv": place(v)}
    dc.dynconv_attn_window_bwd(*ins[:3], o, lse, ins[3], window, sinks=sinks, out=out)
    assert wide.stride(1) * wide.element_size() * (T - 1) > 2 ** 32
    for n, x in {"o": o, "lse": lse, **out}.items():
        assert torch.equal(x, want[n]), n
    assert not wide[:, :, at:].any()


@pytest.mark.parametrize("cu", [None, [0, 77, 200]])
def test_a_window_of_the_whole_row_is_none(cu):
    """Bit for bit the call without a window, from T tokens on."""
    _note(f"[window] whole row {cu}")
    q, k, v, d_o = _row(1, 200, 4, 2, 64, "bf16", seed=3)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, lse = dc.dynconv_attn_fwd(q, k, v, cu_seqlens=c, want_lse=True)
    want = {"o": o, "lse": lse, **dc.dynconv_attn_bwd(q, k, v, o, lse, d_o, cu_seqlens=c)}
    for window in (200, 1000, 2 ** 40):
        got = _run(q, k, v, d_o, window, 3, cu=cu)
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_views():
    """Head-major tensors, heads shared by stride 0, gradients into the parts of one row: bitwise as for plain tensors."""
    _note("[window] views")
    q, k, v, d_o = _row(2, 450, 4, 2, 64, "bf16", seed=9)
    ref = _run(q.contiguous(), k.contiguous(), v.contiguous(), d_o, 50, 4)
    hm = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731  [B, heads, T, head_dim] in memory
    got = _run(hm(q), hm(k), hm(v), hm(d_o), 50, 4)
    assert all(torch.equal(got[n], ref[n]) for n in ref)
    row = torch.full((2, 450, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = {"dq": row[:, :, :4], "dk": row[:, :, 4:6], "dv": row[:, :, 6:]}
    dc.dynconv_attn_window_bwd(q, k, v, ref["o"], ref["lse"], d_o, 50, sinks=4, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], ref[n]) for n in out)
    one_k, one_v = k[:, :, :1].expand(-1, -1, 2, -1), v[:, :, :1].expand(-1, -1, 2, -1)
    got = _run(q, one_k, one_v, d_o, 50, 4)
    ref = _run(q, one_k.contiguous(), one_v.contiguous(), d_o, 50, 4)
    assert all(torch.equal(got[n], ref[n]) for n in ref)


BAD = [math.inf, -math.inf, math.nan, 3.0e38]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H,G", [(600, 4, 2), (4200, 8, 4)])
@pytest.mark.parametrize("hd", [64, 96, 128])
@pytest.mark.parametrize("bad", BAD, ids=str)
def test_what_a_window_leaves_behind_does_not_reach(bad, hd, T, H, G, dtype):
    """Keys and values between the sinks and the window hold what would spoil a product with a zero, and so do another
    document and the padding."""
    _note(f"[window] {bad} behind the window T={T} hd={hd} {dtype}")
    window, sinks, cu = 90, 5, [0, T // 2, T // 2 + 40, T - 20]
    q, k, v, d_o = _row(1, T, H, G, hd, dtype, seed=13)
    want = _run(q, k, v, d_o, window, sinks, cu=cu)
    lo = 20  # tokens 20 .. 59 of the first document: out of sight from token 149 on
    seen = list(range(lo)) + list(range(lo + 40 + window - 1, T // 2))
    q2, k2, v2, d2 = (t.clone() for t in (q, k, v, d_o))
    k2[:, lo:lo + 40] = bad
    v2[:, lo:lo + 40] = bad
    for t in (q2, k2, v2, d2):
        t[:, T // 2:T // 2 + 40] = bad  # the second document
        t[:, T - 20:] = bad             # the padding
    got = _run(q2, k2, v2, d2, window, sinks, cu=cu)
    for n in ("o", "dq"):
        assert torch.equal(got[n][:, seen], want[n][:, seen]), n
        assert bool((got[n][:, T - 20:] == 0).all()), n
    for n in ("dk", "dv"):  # keys that no query of those tokens' sight sees
        far = list(range(lo + 40 + window - 1 + 1, T // 2))
        assert torch.equal(got[n][:, far], want[n][:, far]), n
    for n in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[n][:, T // 2 + 40:T - 20], want[n][:, T // 2 + 40:T - 20]), n
    # gradients of queries that do not see a key: spoilt queries past the window of keys 100 .. 150 (no sinks)
    q3, d3 = q.clone(), d_o.clone()
    q3[:, 260:270] = bad
    d3[:, 260:270] = bad
    got = _run(q3, k, v, d3, window, sinks, cu=cu)
    for n in ("dk", "dv"):
        assert torch.equal(got[n][:, sinks:260 - window + 1], want[n][:, sinks:260 - window + 1]), n
        assert torch.equal(got[n][:, 270:], want[n][:, 270:]), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", BAD[:3], ids=str)
def test_seen_sinks_keep_what_they_hold(bad, dtype):
    """An infinity or a NaN in a sink's value reaches every later token's element, and in a sink's key the far
    queries' gradients as the formulas say: NaN where 0 x infinity is formed; no key out of sight takes part."""
    _note(f"[window] {bad} in a sink {dtype}")
    q, k, v, _ = _row(1, 900, 2, 1, 64, dtype, seed=19)
    v = v.clone()
    v[:, 1, :, 3] = bad
    got = dc.dynconv_attn_window_fwd(q, k, v, 40, sinks=2)
    ref = wu.attention(q, k, v, 40, 2)["o"]
    assert au.rel(got, ref) <= au.TOL[dtype]
    assert bool((~torch.isfinite(got[:, 1:, :, 3])).all()) and bool(torch.isfinite(got[:, :, :, 4:]).all())


@pytest.mark.parametrize("packed", [False, True])
def test_gradients_against_differences(packed):
    """Central differences of sum(o * d_o) along random directions (fp32 outputs, fp64 sums, step 1/64:
    truncation of order step^2, rounding 2^-24 / step)."""
    _note("[window] differences")
    q, k, v, d_o = (t.contiguous() for t in _row(1, 400, 4, 2, 32, "fp32", seed=21))
    cu = [0, 33, 400] if packed else None
    g = _run(q, k, v, d_o, 25, 3, cu=cu)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(22)
    step = 1 / 64
    for name, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        x = [q, k, v]
        d = torch.randn(x[i].shape, generator=gen, device="cuda")

        def loss(sign):
            y = list(x)
            y[i] = x[i] + sign * step * d
            return (dc.dynconv_attn_window_fwd(*y, 25, sinks=3, cu_seqlens=c).double() * d_o.double()).sum()

        num = ((loss(1) - loss(-1)) / (2 * step)).item()
        ana = (g[name].double() * d.double()).sum().item()
        size = g[name].double().norm().item() * math.sqrt(d.numel()) / math.sqrt(g[name].numel()) + 1.0
        assert abs(num - ana) <= 1e-2 * size, (name, num, ana, size)


def test_repeatable_and_on_two_streams():
    _note("[window] repeat, two streams")
    q, k, v, d_o = _row(2, 1700, 8, 2, 128, "bf16", seed=31)
    ref = _run(q, k, v, d_o, 200, 4)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        out = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                o, lse = dc.dynconv_attn_window_fwd(q, k, v, 200, sinks=4, want_lse=True)
                out.append({"o": o, "lse": lse, **dc.dynconv_attn_window_bwd(q, k, v, o, lse, d_o, 200, sinks=4)})
        torch.cuda.synchronize()
        for got in out:
            assert all(torch.equal(got[n], ref[n]) for n in ref)
    s = streams[0]
    s.wait_stream(torch.cuda.current_stream())
    o, lse = dc.dynconv_attn_window_fwd(q, k, v, 200, sinks=4, want_lse=True, stream=s)
    g = dc.dynconv_attn_window_bwd(q, k, v, o, lse, d_o, 200, sinks=4, stream=s)
    s.synchronize()
    assert torch.equal(o, ref["o"]) and all(torch.equal(g[n], ref[n]) for n in g)


def test_graph_replay():
    _note("[window] graph")
    q, k, v, d_o = (t.contiguous() for t in _row(1, 1333, 4, 2, 64, "bf16", seed=41))
    c = torch.tensor([0, 100, 1300], dtype=torch.int32, device="cuda")

    def step():
        o, lse = dc.dynconv_attn_window_fwd(q, k, v, 60, sinks=3, cu_seqlens=c, want_lse=True)
        return {"o": o, "lse": lse, **dc.dynconv_attn_window_bwd(q, k, v, o, lse, d_o, 60, sinks=3, cu_seqlens=c)}

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
        for t, n in zip((q, k, v, d_o), _row(1, 1333, 4, 2, 64, "bf16", seed=50 + r)):
            t.copy_(n)
        c.copy_(torch.tensor([0, 60 + 300 * r, 1333 - r], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], eager[n]) for n in eager), r


def test_empty():
    q = torch.empty(0, 5, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert dc.dynconv_attn_window_fwd(q, q, q, 3).shape == q.shape
    q = torch.empty(2, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = dc.dynconv_attn_window_fwd(q, q, q, 3, sinks=1, want_lse=True)
    g = dc.dynconv_attn_window_bwd(q, q, q, o, lse, q, 3, sinks=1)
    torch.cuda.synchronize()
    assert lse.shape == (2, 4, 0) and g["dk"].shape == q.shape


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [24, 64, 80, 128])
@pytest.mark.parametrize("cu,T", [([0, 130, 100], 130), ([0, 40, 700, 90, 300], 520), ([0, 900, 100, 2000], 1500)],
                         ids=["130", "520", "1500"])
def test_offsets_that_fall_stay_inside_the_row(cu, T, hd, dtype):
    """The tensors end a buffer whose rest holds NaN: a row read past them would show, and none is written."""
    _note(f"[window] falling offsets {cu} {hd} {dtype}")
    H, G = 4, 2
    dt = au.DTYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(5)

    def framed(heads, fill):
        whole = torch.full((T + 256, heads, hd), math.nan, dtype=dt, device="cuda")
        whole[128:128 + T] = fill
        return whole, whole[128:128 + T].unsqueeze(0)

    ins = [framed(h, torch.randn(T, h, hd, generator=g, device="cuda").to(dt)) for h in (H, G, G, H)]
    outs = [framed(h, 7.0) for h in (H, H, G, G)]
    (_, q), (_, k), (_, v), (_, d_o) = ins
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    _, lse = dc.dynconv_attn_window_fwd(q, k, v, 33, sinks=5, cu_seqlens=c, o=outs[0][1], want_lse=True)
    dc.dynconv_attn_window_bwd(q, k, v, outs[0][1], lse, d_o, 33, sinks=5, cu_seqlens=c,
                               out={"dq": outs[1][1], "dk": outs[2][1], "dv": outs[3][1]})
    torch.cuda.synchronize()
    for whole, _ in ins + outs:
        assert bool(torch.isnan(whole[:128]).all()) and bool(torch.isnan(whole[128 + T:]).all())
    assert bool(torch.isfinite(outs[0][1]).all()) and bool(torch.isfinite(outs[1][1]).all())


def _off_over_own(got, ref):
    """The error over that of rounding the exact result to bf16."""
    own = (ref.bfloat16().double() - ref).norm().item()
    return (got.double() - ref).norm().item() / own if own else 0.0


@pytest.mark.parametrize("H,G,hd", [(4, 2, 64), (4, 2, 128), (6, 2, 96)])
@pytest.mark.parametrize("B,T,window,sinks", [(1, 300, 2, 0), (1, 300, 3, 1), (20, 300, 16, 2), (2, 1000, 60, 4), (1, 1000, 1, 63)])
def test_few_keys_in_bf16_lose_no_more_than_their_own_rounding(B, T, window, sinks, H, G, hd):
    """Windows and sinks of up to 64 keys keep 16 bits of p and ds (2^-17 relative) and take delta from the
    products themselves: what is left beside the outputs' own rounding is fp32 sums, far below it.  1.1: the
    error of two independent roundings of which one is 0.4 of the other."""
    _note(f"[window] few keys B={B} T={T} window {window} sinks {sinks} hd={hd}")
    q, k, v, d_o = _row(B, T, H, G, hd, "bf16", seed=T + window)
    got, ref = _run(q, k, v, d_o, window, sinks), wu.attention(q, k, v, window, sinks, d_o=d_o)
    off = {n: _off_over_own(got[n], ref[n]) for n in ("o", "dq", "dk", "dv")}
    assert all(x <= 1.1 for x in off.values()), off


def test_autograd_of_the_path():
    """QKVAttnFn with a window: o and the gradient of the row against autograd of the definition in fp64."""
    _note("[window] QKVAttnFn")
    H, G, hd, T, cu, window, sinks = 4, 2, 64, 331, [0, 50, 331], 40, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    row = torch.randn(1, T, (H + 2 * G) * hd, generator=g, device="cuda").requires_grad_()
    d_o = torch.randn(1, T, H, hd, generator=g, device="cuda")
    f = dc.dynconv_rope_freqs(hd)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = dc.QKVAttnFn.apply(row, H, G, f, False, 1.0, None, c, window, sinks)
    o.backward(d_o)
    x = row.detach().double().view(1, T, H + 2 * G, hd)
    pos = torch.cat([torch.arange(b - a) for a, b in zip(cu, cu[1:])]).cuda()[None]
    qk = au.rotate(x[:, :, :H + G].cpu(), f.cpu(), pos.cpu()).cuda()
    ref = wu.attention(qk[:, :, :H], qk[:, :, H:], x[:, :, H + G:], window, sinks, cu=cu, d_o=d_o)
    assert au.rel(o, ref["o"]) <= au.TOL["fp32"]
    back = au.rotate(torch.cat((ref["dq"], ref["dk"]), 2).cpu(), f.cpu(), pos.cpu(), inverse=True).cuda()
    want = torch.cat((back, ref["dv"]), 2).view(1, T, -1)
    assert au.rel(row.grad, want) <= au.TOL["fp32"]


# As many documents as make a short row on average, one of them long.
SHORT_ON_AVERAGE = [0, 600] + list(range(605, 701, 5))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", BAD[:3], ids=str)
@pytest.mark.parametrize("hd", [64, 80, 128])
@pytest.mark.parametrize("window,sinks,cu", [(40, 3, None), (1, 63, None), (200, 4, None), (130, 128, None),
                                             (200, 4, SHORT_ON_AVERAGE)], ids=["40-3", "1-63", "200-4", "130-128", "packed"])
def test_far_gradients_that_are_not_finite(window, sinks, cu, hd, bad, dtype):
    """Infinities and NaN in d_o of queries that see the sinks past the window: the sinks' dv holds them as the formula
    does, with their sign (and their dk NaN: the query's d_o.v and d_o.o are the same infinity)."""
    _note(f"[window] {bad} in d_o past the window {window} {sinks} hd={hd} {dtype}")
    q, k, v, d_o = _row(1, 700, 4, 2, hd, dtype, seed=23)
    v, d_o = v.clone(), d_o.clone()
    v[..., 3], v[..., 5] = v[..., 3].abs() + 0.25, v[..., 5].abs() + 0.25
    d_o[:, 520, 1, 3], d_o[:, 531, 2, 5] = bad, -bad
    got, ref = _run(q, k, v, d_o, window, sinks, cu=cu), wu.attention(q, k, v, window, sinks, cu=cu, d_o=d_o)
    if not math.isnan(bad):
        assert bool((ref["dv"][:, :sinks, 0, 3] == bad).all()) and bool((ref["dv"][:, :sinks, 1, 5] == -bad).all())
    errs = {n: au.rel(got[n], ref[n]) for n in ("o", "dq", "dk", "dv")}
    assert all(e <= au.TOL[dtype] for e in errs.values()), errs


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(40, 3), (200, 4)])
def test_gradients_of_a_sink_without_weight(window, sinks, dtype):
    """A sink's key of -infinity where every query is positive: its weight is 0 everywhere, its own dk and dv are 0, and dq
    holds the NaN of 0 x infinity in that element."""
    _note(f"[window] -infinity in a sink's key {window} {sinks} {dtype}")
    q, k, v, d_o = _row(1, 700, 4, 2, 64, dtype, seed=27)
    q, k = q.clone(), k.clone()
    q[..., 3] = q[..., 3].abs() + 0.25
    k[:, 1, 0, 3] = -math.inf
    got, ref = _run(q, k, v, d_o, window, sinks), wu.attention(q, k, v, window, sinks, d_o=d_o)
    errs = {n: au.rel(got[n], ref[n]) for n in ("o", "dq", "dk", "dv")}
    assert all(e <= au.TOL[dtype] for e in errs.values()), errs
    assert bool((got["dk"][:, 1, 0] == 0).all()) and bool((got["dv"][:, 1, 0] == 0).all())
