"""The one-token step over a cache (dynconv_attn_decode) against its fp64
definition: lengths from 0 to the capacity, idle and full slots, grouped heads
(more than 16 to a group among them), stretches of long caches, views, what lies
in cache rows past the length, agreement with the whole-sequence call."""
from __future__ import annotations

import math
import sys

import pytest
import torch

import input_dependent_depthwise_amd as dc
from tests import attn_util as au

pytestmark = pytest.mark.gpu

# bf16: the output's rounding, and the stored key's double rounding against the definition's (2^-8 each);
# fp32: as the rest of the library
TOL = {"bf16": 2 * 2.0 ** -8, "fp32": 1e-5}


def _note(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _inputs(B, S, H, G, hd, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(au.DTYPES[dtype])  # noqa: E731
    row = r(B, H + 2 * G, hd)
    return row[:, :H], row[:, H:H + G], row[:, H + G:], r(B, S, G, hd), r(B, S, G, hd)


def _check(shape, lengths, dtype, **kw):
    B, S, H, G, hd = shape
    q, k, v, kc, vc = _inputs(B, S, H, G, hd, dtype, seed=S + H + hd)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ro, rk, rv = au.decode(q, k, v, kc, vc, n, **kw)
    for b, m in enumerate(lengths):  # rows past the length are never read
        if m >= 0:
            kc[b, m:], vc[b, m:] = math.nan, math.inf
    before = kc.clone(), vc.clone()
    o = dc.dynconv_attn_decode(q, k, v, kc, vc, n, **kw)
    torch.cuda.synchronize()
    assert au.rel(o, ro) <= TOL[dtype]
    for got, ref, old in ((kc, rk, before[0]), (vc, rv, before[1])):
        for b, m in enumerate(lengths):
            rest = torch.ones(S, dtype=torch.bool, device="cuda")
            if 0 <= m < S:
                assert au.rel(got[b, m], ref[b, m]) <= (2.0 ** -8 if dtype == "bf16" else 1e-6)
                rest[m] = False
            assert torch.equal(got[b, rest].nan_to_num(), old[b, rest].nan_to_num())
    for b, m in enumerate(lengths):
        if m < 0 or m >= S:
            assert bool((o[b] == 0).all())


CASES = [
    # (B, capacity, H, G, hd), lengths
    ((1, 1, 1, 1, 64), [0]),
    ((3, 4, 4, 2, 128), [0, 3, 4]),
    ((4, 40, 4, 4, 16), [31, 32, 33, -1]),
    ((2, 300, 8, 1, 80), [255, 299]),
    ((2, 300, 6, 3, 96), [256, 257]),
    ((2, 700, 12, 12, 64), [699, 1]),
    ((1, 1024, 40, 2, 64), [1000]),
    ((3, 3000, 16, 4, 128), [2999, 0, 1500]),
    ((2, 5000, 34, 1, 128), [4999, 257]),
    ((5, 2100, 2, 1, 8), [2099, 1023, 1024, 1025, -5]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[0])))
def test_against_definition(case, dtype):
    _note(f"[decode] {case} {dtype}")
    _check(*case, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("rot", [128, 64, 10])
def test_rotated(rot, interleaved, dtype):
    _note(f"[decode] rot={rot} interleaved={interleaved} {dtype}")
    f = dc.dynconv_rope_freqs(rot)
    _check((3, 2000, 8, 2, 128), [1999, 0, 700], dtype, freqs=f, interleaved=interleaved, factor=1.1)


def test_scale():
    _check((2, 500, 4, 2, 64), [400, 499], "fp32", scale=0.5)


def test_views():
    """Head-major caches and both caches in one buffer: bitwise as for plain ones."""
    _note("[decode] views")
    q, k, v, kc, vc = _inputs(2, 900, 8, 2, 64, "bf16", seed=7)
    n = torch.tensor([880, 33], dtype=torch.int32, device="cuda")
    k0, v0 = kc.clone(), vc.clone()
    ref = dc.dynconv_attn_decode(q, k, v, k0, v0, n)
    hk, hv = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kc, vc))
    both = torch.stack((kc, vc), 2)
    for a, b in ((hk, hv), (both[:, :, 0], both[:, :, 1])):
        o = dc.dynconv_attn_decode(q, k, v, a, b, n)
        torch.cuda.synchronize()
        assert torch.equal(o, ref) and torch.equal(a, k0) and torch.equal(b, v0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_steps_follow_the_prompt(dtype):
    """Rotary, then whole-sequence attention over T tokens; the same tokens one step at a time."""
    _note(f"[decode] steps {dtype}")
    B, T, H, G, hd = 2, 40, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(11)
    row = torch.randn(B, T, H + 2 * G, hd, generator=g, device="cuda").to(au.DTYPES[dtype])
    f = dc.dynconv_rope_freqs(hd)
    qk = dc.dynconv_rope(row[:, :, :H + G], f)
    o = dc.dynconv_attn_fwd(qk[:, :, :H], qk[:, :, H:], row[:, :, H + G:])
    kc, vc = (torch.zeros(B, 64, G, hd, dtype=row.dtype, device="cuda") for _ in range(2))
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    steps = []
    for t in range(T):
        x = row[:, t]
        steps.append(dc.dynconv_attn_decode(x[:, :H], x[:, H:H + G], x[:, H + G:], kc, vc, n, freqs=f))
        n += 1
    assert torch.equal(kc[:, :T], qk[:, :, H:])
    # the prompt's turned queries are rounded to bf16, the step's are not: one more rounding each of q and p
    assert au.rel(torch.stack(steps, 1), o) <= (4 * 2.0 ** -8 if dtype == "bf16" else 1e-5)


def test_graph_replay():
    _note("[decode] graph")
    q, k, v, kc, vc = _inputs(2, 2048, 8, 2, 64, "bf16", seed=17)
    q, k, v = (t.contiguous() for t in (q, k, v))
    n = torch.tensor([0, 1500], dtype=torch.int32, device="cuda")
    f = dc.dynconv_rope_freqs(64)
    step = lambda a, b, m: dc.dynconv_attn_decode(q, k, v, a, b, m, freqs=f)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(kc, vc, n)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(kc, vc, n)
        n.add_(1)
    k0, v0, n0 = kc.clone(), vc.clone(), n.clone()
    for r in range(4):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = step(k0, v0, n0)
        n0.add_(1)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(kc, k0) and torch.equal(vc, v0) and torch.equal(n, n0), r


def test_empty_batch():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.empty(0, 16, 4, 64, dtype=torch.bfloat16, device="cuda")
    n = torch.empty(0, dtype=torch.int32, device="cuda")
    assert dc.dynconv_attn_decode(q, q, q, kc, kc.clone(), n).shape == q.shape


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("S,n", [(1, 0), (40, 39), (40, 12), (700, 600), (5000, 4900)])
@pytest.mark.parametrize("hd", [64, 96, 128])
def test_seen_infinities(hd, S, n, dtype):
    """Infinities and NaN in rows that are read, as in the sums themselves: a value of +infinity makes its
    element +infinity; a key whose score is -infinity has no weight; a NaN, or +infinity and -infinity in one
    element, makes that a NaN; a score of +infinity a head's whole row."""
    _note(f"[decode] seen infinities {hd} {S} {n} {dtype}")
    B, H, G = 2, 6, 2
    q, k, v, kc, vc = (t.clone() for t in _inputs(B, S, H, G, hd, dtype, seed=S + hd))
    q[:, :, 3] = q[:, :, 3].abs() + 0.25
    q[:, :, 9] = -q[:, :, 9].abs() - 0.25
    v[0, :, 0], v[0, 0, 1], v[1, 1, 2] = math.inf, -math.inf, math.nan
    if n > 8:
        vc[:, 4, 0, 5], vc[:, 7, 1, 6], vc[0, 2, :, 7], vc[0, 8, :, 7] = math.inf, -math.inf, math.inf, -math.inf
        vc[1, 3, 1, 8] = math.nan
        kc[:, 5, 0, 3], kc[:, 6, 1, 9], kc[:, 1, :, 3] = -math.inf, math.inf, -math.inf
        k[1, :, 3] = -math.inf  # the new key of one sequence has no weight (and its NaN value no finite product)
        v[1] = 1.0
        q[1, 5, 4] = math.inf   # one head's scores are all infinite
    lengths = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    ro, _, _ = au.decode(q, k, v, kc, vc, lengths)
    o = dc.dynconv_attn_decode(q, k, v, kc, vc, lengths)
    torch.cuda.synchronize()
    assert au.rel(o, ro) <= TOL[dtype]
    assert bool((o[0, :, 0] == math.inf).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape,lengths", [((3, 40, 4, 2, 64), [31, 0, -1]), ((2, 3000, 6, 2, 96), [2500, 3000]),
                                           ((1, 5000, 8, 1, 128), [4097])], ids=["40", "3000", "5000"])
def test_no_other_cache_row_is_written(shape, lengths, dtype):
    """Bit for bit, NaN of every payload among them (a zero written over a NaN would show)."""
    _note(f"[decode] other rows {shape} {lengths} {dtype}")
    B, S, H, G, hd = shape
    q, k, v, kc, vc = _inputs(*shape, dtype, seed=S)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    g = torch.Generator(device="cuda").manual_seed(S)
    for c in (kc, vc):
        for b, n in enumerate(lengths):
            if n >= 0:  # rows that are not read hold any bits
                c[b, n:].view(bits).random_(generator=g)
    before = kc.view(bits).clone(), vc.view(bits).clone()
    dc.dynconv_attn_decode(q, k, v, kc, vc, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for c, old, new in ((kc, before[0], k), (vc, before[1], v)):
        want = old.clone()
        for b, n in enumerate(lengths):
            if 0 <= n < S:
                want[b, n] = new.view(bits)[b]
        assert torch.equal(c.view(bits), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("S,n", [(1, 0), (60, 40), (5000, 4000)])
def test_scores_that_are_all_minus_infinity(S, n, dtype):
    """A row without any weight is zero, as in the whole-sequence call; the other heads keep theirs."""
    _note(f"[decode] all -infinity {S} {n} {dtype}")
    H, G, hd = 4, 2, 64
    q, k, v, kc, vc = (t.clone() for t in _inputs(1, S, H, G, hd, dtype, seed=S))
    q[:, :2, 3] = 1.0
    k[:, 0, 3], kc[:, :, 0, 3] = -math.inf, -math.inf
    keys, values = torch.cat((kc[:, :n], k[:, None]), 1), torch.cat((vc[:, :n], v[:, None]), 1)
    o = dc.dynconv_attn_decode(q, k, v, kc, vc, torch.tensor([n], dtype=torch.int32, device="cuda"))
    rows = q[:, None].expand(-1, n + 1, -1, -1).contiguous()
    want, lse = dc.dynconv_attn_fwd(rows, keys, values, want_lse=True)
    torch.cuda.synchronize()
    assert bool((want[:, -1, :2] == 0).all()) and bool((lse[:, :2] == -math.inf).all())
    assert bool((o[:, :2] == 0).all())
    assert au.rel(o[:, 2:], want[:, -1, 2:].double()) <= (4 * 2.0 ** -8 if dtype == "bf16" else 1e-5)
