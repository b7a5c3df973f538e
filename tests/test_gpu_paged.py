"""A cache kept in pages: storing prompts (dynconv_attn_paged_store) and the one-token step over it
(dynconv_attn_paged_decode) against plain fp64 definitions: pages of any size, lists with missing, wrong and shared
pages, windows with sinks, ragged batches that are split and joined, what is not read holding NaN, what is not
written keeping its bits, graphs, streams, views, pools past 4 GiB."""
from __future__ import annotations

import math
import sys

import pytest
import torch

import input_dependent_depthwise_amd as dc
from tests import attn_util as au
from tests import window_util as wu

pytestmark = pytest.mark.gpu

# o: its own rounding (2^-8 for bf16, half a step), q and p enter with 16 bits or more; fp32: sums of some thousand terms.
TOL = {"bf16": 2.0 ** -8 + 1e-4, "fp32": 1e-5}


def _note(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def _cache(lengths, per_seq, size, G, hd, dtype, seed, spare=3):
    """Pools whose rows below each length hold numbers and all others NaN, and the table (pages in random order, -1 past
    those in use, the new token's among them)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [0 if n < 0 else min(per_seq, n // size + 1) for n in lengths]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((len(lengths), per_seq), -1, dtype=torch.int32, device="cuda")
    kp, vp = (torch.full((n_pages, size, G, hd), math.nan, dtype=au.DTYPES[dtype], device="cuda") for _ in range(2))
    at = 0
    for b, (n, m) in enumerate(zip(lengths, need)):
        table[b, :m] = order[at:at + m]
        at += m
        if n > 0:
            j = torch.arange(min(n, per_seq * size), device="cuda")
            rows = table[b].long()[j // size] * size + j % size
            for pool in (kp, vp):
                pool.flatten(0, 1)[rows] = torch.randn(len(j), G, hd, generator=g, device="cuda").to(pool.dtype)
    return kp, vp, table


def _new(B, H, G, hd, dtype, seed):
    row = torch.randn(B, H + 2 * G, hd, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    row = row.to(au.DTYPES[dtype])
    return row[:, :H], row[:, H:H + G], row[:, H + G:]


def _step(lengths, per_seq, size, H, G, hd, dtype, window=None, sinks=0, seed=1, cache=None, tol=None, **kw):
    """A step against its definition; the stored rows, and every other row's bits.  Returns o."""
    B = len(lengths)
    kp, vp, table = cache or _cache(lengths, per_seq, size, G, hd, dtype, seed)
    q, k, v = _new(B, H, G, hd, dtype, seed + 1)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    before = kp.clone(), vp.clone()
    o = dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, n, window=window, sinks=sinks, **kw)
    torch.cuda.synchronize()
    rot = {x: y for x, y in kw.items() if x in ("freqs", "interleaved", "factor")}
    want_k = k.double()
    if "freqs" in kw:
        want_k = au.rotate(k[:, None].cpu(), kw["freqs"].cpu(), n.view(B, 1).cpu(), kw.get("interleaved", False),
                           kw.get("factor", 1.0))[:, 0].cuda()
    got_k, want_kp, want_vp = want_k.clone(), before[0].clone(), before[1].clone()
    for b, m in enumerate(lengths):
        if 0 <= m < per_seq * size:
            rows, ok = wu.paged_rows(table, kp.shape[0], size, b, torch.tensor([m], device="cuda"))
            if bool(ok):
                got_k[b] = kp.flatten(0, 1)[rows[0]].double()
                want_kp.flatten(0, 1)[rows[0]] = kp.flatten(0, 1)[rows[0]]
                want_vp.flatten(0, 1)[rows[0]] = v[b]
    # the turned key: fp32 arithmetic, then one rounding
    off = (got_k - want_k).abs() - (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22) * want_k.abs()
    assert bool((off <= 1e-6).all())
    assert torch.equal(_bits(kp), _bits(want_kp)) and torch.equal(_bits(vp), _bits(want_vp))
    ref = wu.paged_decode(q, got_k.to(q.dtype), v, *before, table, n, window, sinks, kw.get("scale"), **rot)
    err = au.rel(o, ref)
    assert err <= (tol or TOL[dtype]), err
    for b, m in enumerate(lengths):
        if m < 0 or m >= per_seq * size:
            assert bool((o[b] == 0).all())
    return o


CASES = [
    # lengths, pages a list, page size, H, G, hd
    ([0], 1, 1, 1, 1, 64),
    ([0, 3, -1, 5], 6, 1, 4, 2, 64),
    ([16, 15, 47, 48], 3, 16, 12, 12, 64),      # a full list: idle
    ([33, 64, 65, 31], 20, 5, 6, 2, 128),
    ([100, 7], 9, 13, 7, 1, 80),
    ([250, -5, 0, 1 << 30], 4, 64, 17, 1, 96),   # more than 16 query heads to a key head
    ([129], 1, 200, 40, 2, 8),
    ([1000, 40, 700], 64, 16, 8, 2, 16),
    ([3000, 1, 2999, 513, -1], 200, 16, 16, 4, 128),
    ([5000], 700, 8, 12, 12, 64),
    ([9000, 100], 300, 32, 4, 1, 128),
    ([2100, 2400, 3], 60, 40, 34, 2, 64),
    ([4000, 2400, 0, 3999], 101, 40, 34, 2, 64),  # column blocks of 16 and 1 heads
    ([3300, 70], 250, 16, 5, 5, 104),
    ([3500, 3100, 900], 500, 8, 14, 14, 24),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{c[1]}x{c[2]}-{c[3]}-{c[4]}-{c[5]}")
def test_against_definition(case, dtype):
    lengths, per_seq, size, H, G, hd = case
    _note(f"[paged] {case} {dtype}")
    _step(lengths, per_seq, size, H, G, hd, dtype)


WINDOWS = [(1, 0), (1, 3), (2, 1), (31, 4), (33, 33), (64, 128), (700, 4), (10 ** 9, 5)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("size,hd", [(16, 64), (5, 128)])
def test_window(size, hd, window, sinks, dtype):
    lengths = [0, 1, 30, 64, 1500, 2000, -1, 65]
    _note(f"[paged] window {window} sinks {sinks} pages of {size} {hd} {dtype}")
    _step(lengths, 2040 // size, size, 4, 2, hd, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(3400, 4), (3400, 128), (5000, 33)])
@pytest.mark.parametrize("size,H,G,hd", [(16, 4, 2, 64), (7, 3, 3, 128), (64, 20, 1, 96)])
def test_long_window(size, H, G, hd, window, sinks, dtype):
    """Windows long enough that a sequence is shared among blocks."""
    lengths = [0, 3399, 3401, 5950, -1, 6000, 5000, 40]
    _note(f"[paged] window {window} sinks {sinks} pages of {size} {H} {G} {hd} {dtype}")
    _step(lengths, 6100 // size, size, H, G, hd, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True), (10, False), (10, True)])
def test_rotated(rot, interleaved, dtype):
    _note(f"[paged] rotated {rot} {interleaved} {dtype}")
    f = dc.dynconv_rope_freqs(rot)
    _step([0, 77, 300], 40, 8, 4, 2, 128, dtype, freqs=f, interleaved=interleaved, factor=1.2)
    _step([2000, 77, 300], 300, 8, 4, 2, 128, dtype, window=90, sinks=3, freqs=f, interleaved=interleaved)


def test_scale():
    # scores of some tens: an fp32 score error of |s| 2^-22 or so is far below the output's rounding
    _step([100, 900], 64, 16, 4, 2, 64, "bf16", scale=2.0, tol=2.0 ** -8 + 1e-3)


BAD = [-1, -2 ** 31, 2 ** 31 - 1, None]  # None: one past the pool


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", BAD, ids=str)
@pytest.mark.parametrize("lengths,per_seq", [([100, 61, 40], 8), ([2500, 61, 1500], 200)], ids=["short", "long"])
def test_pages_that_are_none(lengths, per_seq, bad, dtype):
    """Their tokens are not seen, and a new token without a page is seen but not stored."""
    _note(f"[paged] bad pages {bad} {lengths} {dtype}")
    size = 16
    kp, vp, table = _cache(lengths, per_seq, size, 2, 64, dtype, 4)
    bad = kp.shape[0] if bad is None else bad
    table[0, 2] = table[0, 5] = bad
    table[1, lengths[1] // size] = bad  # the new token's (and those cached beside it)
    table[2, :] = bad                   # a sequence without any
    table[:, lengths[0] // size + 1:] = bad
    _step(lengths, per_seq, size, 6, 2, 64, dtype, cache=(kp, vp, table))
    _step(lengths, per_seq, size, 6, 2, 64, dtype, 70, 20, cache=(kp, vp, table))


def test_what_a_window_left_behind_may_be_given_back():
    """Pages between the sinks and the window, by other entries or none: bit for bit the same."""
    _note("[paged] given back")
    lengths, size = [3000, 1700], 16
    kp, vp, table = _cache(lengths, 200, size, 2, 128, "bf16", 6)
    q, k, v = _new(2, 8, 2, 128, "bf16", 7)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    args = dict(window=500, sinks=4)
    want = dc.dynconv_attn_paged_decode(q, k, v, kp.clone(), vp.clone(), table, n, **args)
    free = table.clone()
    for b, m in enumerate(lengths):
        free[b, 1:(m + 1 - 500) // size] = -1
    got = dc.dynconv_attn_paged_decode(q, k, v, kp.clone(), vp.clone(), free, n, **args)
    other = torch.where(free < 0, table.flip(0), free)
    again = dc.dynconv_attn_paged_decode(q, k, v, kp.clone(), vp.clone(), other, n, **args)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)


def test_shared_pages():
    """Two sequences with the same first pages, and one that lists a page twice."""
    _note("[paged] shared")
    size, lengths = 8, [70, 66, 66]
    kp, vp, table = _cache(lengths, 12, size, 2, 64, "fp32", 8)
    table[1, :6] = table[0, :6]
    table[2, 3] = table[2, 1]
    _step(lengths, 12, size, 4, 2, 64, "fp32", cache=(kp, vp, table))


def test_pages_as_the_dense_cache():
    """Pages of a dense cache in order: the same attention as the call over the cache itself (its sums are split in another way)."""
    _note("[paged] dense")
    B, S, H, G, hd, size = 3, 512, 8, 2, 128, 32
    g = torch.Generator(device="cuda").manual_seed(9)
    kc, vc = (torch.randn(B, S, G, hd, generator=g, device="cuda") for _ in range(2))
    q, k, v = _new(B, H, G, hd, "fp32", 10)
    n = torch.tensor([511, 100, 0], dtype=torch.int32, device="cuda")
    table = torch.arange(B * S // size, dtype=torch.int32, device="cuda").view(B, -1)
    kp, vp = kc.clone().view(-1, size, G, hd), vc.clone().view(-1, size, G, hd)
    f = dc.dynconv_rope_freqs(hd)
    o = dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, n, freqs=f)
    want = dc.dynconv_attn_decode(q, k, v, kc, vc, n, freqs=f)
    torch.cuda.synchronize()
    assert torch.equal(kp.view_as(kc), kc) and torch.equal(vp.view_as(vc), vc)
    assert au.rel(o, want) <= TOL["fp32"]


def test_views():
    """Head-major pools, k and v pages that alternate in one buffer, a table that is a part of a wider one, o in a row."""
    _note("[paged] views")
    lengths, size, G, hd, H = [900, 1300, -1], 16, 2, 64, 4
    kp, vp, table = _cache(lengths, 100, size, G, hd, "bf16", 11)
    q, k, v = _new(3, H, G, hd, "bf16", 12)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want = dc.dynconv_attn_paged_decode(q, k, v, kp.clone(), vp.clone(), table, n)
    hm = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    both = torch.stack((kp, vp), 1)
    wide = torch.full((3, 150), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, 20:120] = table
    row = torch.full((3, 9, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    a = dc.dynconv_attn_paged_decode(q, k, v, hm(kp), hm(vp), table, n)
    b = dc.dynconv_attn_paged_decode(q, k, v, both[:, 0], both[:, 1], wide[:, 20:120], n, o=row[:, 3:3 + H])
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    assert bool((row[:, :3] == 7).all()) and bool((row[:, 3 + H:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [0, 40, 4000])
@pytest.mark.parametrize("hd", [64, 96, 128])
def test_seen_infinities(hd, n, dtype):
    """Infinities and NaN in rows that are read, as in the sums themselves."""
    _note(f"[paged] seen infinities {hd} {n} {dtype}")
    H, G, size = 6, 2, 16
    kp, vp, table = _cache([n, n], 300, size, G, hd, dtype, n + hd)
    q, k, v = (t.clone() for t in _new(2, H, G, hd, dtype, 3))
    q[:, :, 3] = q[:, :, 3].abs() + 0.25
    q[:, :, 9] = -q[:, :, 9].abs() - 0.25
    v[0, :, 0], v[0, 0, 1], v[1, 1, 2] = math.inf, -math.inf, math.nan
    if n:
        row = lambda b, j: int(table[b, j // size]) * size + j % size  # noqa: E731
        kf, vf = kp.flatten(0, 1), vp.flatten(0, 1)
        vf[row(0, 4), 0, 5], vf[row(0, 7), 1, 6], vf[row(0, 2), :, 7], vf[row(0, 8), :, 7] = math.inf, -math.inf, math.inf, -math.inf
        vf[row(1, 3), 1, 8] = math.nan
        kf[row(0, 5), 0, 3], kf[row(0, 6), 1, 9], kf[row(1, 1), :, 3] = -math.inf, math.inf, -math.inf
        k[1, :, 3] = -math.inf
        v[1] = 1.0
        q[1, 5, 4] = math.inf
    lengths = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    ref = wu.paged_decode(q, k, v, kp, vp, table, lengths)
    o = dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, lengths)
    torch.cuda.synchronize()
    assert au.rel(o, ref) <= TOL[dtype]
    assert bool((o[0, :, 0] == math.inf).all())


@pytest.mark.parametrize("B", [40, 1000])
def test_seen_infinities_among_many(B):
    """A block takes several sequences one after another: one that starts over (an infinity among its values, behind its
    first groups) leaves the next one as it is."""
    _note(f"[paged] infinities among {B}")
    lengths = [100, 40] * (B // 2)
    kp, vp, table = _cache(lengths, 250, 16, 2, 64, "bf16", B)
    for b in range(0, B, 2):
        vp[int(table[b, 6]), 2, :, 5] = math.inf  # token 98
    q, k, v = _new(B, 4, 2, 64, "bf16", B + 1)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ref = wu.paged_decode(q, k, v, kp, vp, table, n)
    o = dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, n)
    torch.cuda.synchronize()
    assert au.rel(o, ref) <= TOL["bf16"]


@pytest.mark.parametrize("n", [0, 40, 4000])
def test_scores_that_are_all_minus_infinity(n):
    _note(f"[paged] all -infinity {n}")
    kp, vp, table = _cache([n], 300, 16, 2, 64, "bf16", 5)
    q, k, v = (t.clone() for t in _new(1, 4, 2, 64, "bf16", 6))
    q[:, :2, 3] = 1.0
    k[:, 0, 3] = -math.inf
    kp[:, :, 0, 3] = -math.inf
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    ref = wu.paged_decode(q, k, v, kp, vp, table, lengths)
    o = dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, lengths)
    torch.cuda.synchronize()
    assert bool((o[:, :2] == 0).all()) and au.rel(o, ref) <= TOL["bf16"]


@pytest.mark.parametrize("B", [300, 1030])
def test_large_batches(B):
    """Lengths of all kinds in a batch that is flattened (to 1024 sequences) or not."""
    _note(f"[paged] batch of {B}")
    r = torch.Generator().manual_seed(B)
    lengths = [int(x) for x in (torch.rand(B, generator=r) ** 6 * 3000).long()]
    lengths[5], lengths[B - 1], lengths[0] = -1, 2999, 0
    _step(lengths, 120, 32, 4, 2, 64, "bf16")  # (lists long enough for the flat launch)


def test_one_long_among_short():
    _note("[paged] one long")
    _step([3] * 20 + [60000] + [1] * 20, 4000, 16, 4, 1, 128, "bf16")


def test_no_sequence_at_all():
    """Every slot idle, flattened and not."""
    _note("[paged] idle")
    for per_seq in (2, 400):
        _step([-1, -7, per_seq * 16], per_seq, 16, 4, 2, 64, "bf16")


def test_empty_batch():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    pool = torch.empty(3, 16, 4, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.empty(0, 5, dtype=torch.int32, device="cuda")
    n = torch.empty(0, dtype=torch.int32, device="cuda")
    assert dc.dynconv_attn_paged_decode(q, q, q, pool, pool.clone(), table, n).shape == q.shape
    dc.dynconv_attn_paged_store(q[None], q[None], pool, pool.clone(), torch.zeros(1, 5, dtype=torch.int32, device="cuda"))


# --- storing prompts -----------------------------------------------------------------------------


def _store_case(T, B, G, hd, size, per_seq, dtype, starts, counts, cu, freqs, interleaved, seed, table=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = au.DTYPES[dtype]
    row = torch.randn(B, T, 3 * G, hd, generator=g, device="cuda").to(dt)
    k, v = row[:, :, G:2 * G], row[:, :, 2 * G:]
    lists = len(cu) - 1 if cu else B
    n_pages = lists * per_seq + 2
    if table is None:
        table = torch.randperm(n_pages, generator=g, device="cuda")[:lists * per_seq].int().view(lists, per_seq)
    kp, vp = (torch.empty(n_pages, size, G, hd, dtype=dt, device="cuda") for _ in range(2))
    for pool in (kp, vp):
        _bits(pool).random_(generator=g)
    want_k, want_v = kp.clone(), vp.clone()
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    stored = dc.dynconv_attn_paged_store(k, v, kp, vp, table, starts=i32(starts), counts=i32(counts), cu_seqlens=i32(cu),
                                         freqs=freqs, interleaved=interleaved, factor=1.1 if freqs is not None else 1.0)
    torch.cuda.synchronize()
    assert stored[0] is kp and stored[1] is vp
    # the same one token at a time: turned by the rotary call at its position
    pos = torch.zeros(B, T, dtype=torch.int32)
    place = []
    for b in range(B):
        for t in range(T):
            seq, i = b, t
            if cu:
                seq = next((s for s in range(lists) if cu[s] <= t < cu[s + 1]), None)
                if seq is None:
                    continue
                i = t - cu[seq]
            s = starts[seq] if starts else 0
            if s < 0 or (counts and i >= counts[seq]) or s + i >= per_seq * size:
                continue
            page = int(table[seq, (s + i) // size])
            if 0 <= page < n_pages:
                pos[b, t] = s + i
                place.append((b, t, page * size + (s + i) % size))
    turned = k if freqs is None else dc.dynconv_rope(k, freqs, positions=pos.cuda(), interleaved=interleaved, factor=1.1)
    for b, t, r in place:
        _bits(want_k).flatten(0, 1)[r] = _bits(turned[b, t].contiguous())
        _bits(want_v).flatten(0, 1)[r] = _bits(v[b, t].contiguous())
    assert torch.equal(_bits(kp), _bits(want_k)) and torch.equal(_bits(vp), _bits(want_v))
    return len(place)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rot,interleaved", [(None, False), (64, False), (64, True), (20, False), (8, True), (6, False), (2, True)])
@pytest.mark.parametrize("hd,size", [(64, 16), (104, 5)])
def test_store(hd, size, rot, interleaved, dtype):
    """Bit for bit the rotary call's keys and the values, nothing else touched; starts, counts, idle sequences, full lists."""
    _note(f"[paged] store {hd} pages of {size} rot {rot} {interleaved} {dtype}")
    f = None if rot is None else dc.dynconv_rope_freqs(rot)
    assert _store_case(37, 3, 2, hd, size, 60 // size, dtype, None, None, None, f, interleaved, 1) == 3 * 37
    assert _store_case(50, 4, 3, hd, size, 80 // size, dtype, [0, 17, -1, 70], [50, 8, 50, 50], None, f, interleaved, 2) < 150
    assert _store_case(1, 2, 1, hd, size, 3, dtype, [2, 0], [0, 5], None, f, interleaved, 3) == 1
    n = _store_case(90, 1, 2, hd, size, 100 // size, dtype, [0, 5, 9, -2], None, [0, 0, 31, 80, 85], f, interleaved, 4)
    assert n == 80


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_store_where_there_is_no_page(dtype):
    _note(f"[paged] store, bad pages {dtype}")
    f = dc.dynconv_rope_freqs(64)
    table = torch.tensor([[3, -1, 7, 2 ** 31 - 1], [0, 1, 2, 10], [-2 ** 31, -2 ** 31, -1, -1]], dtype=torch.int32, device="cuda")
    # (12 + 2 pages)
    assert _store_case(64, 3, 2, 64, 16, 4, dtype, [0, 3, 0], None, None, f, False, 5, table=table) == 32 + 61


def test_store_large_and_head_major():
    """Many blocks, pools with the heads outside the rows."""
    _note("[paged] store large")
    T, G, hd, size = 5000, 4, 128, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    row = torch.randn(1, T, 2 * G, hd, generator=g, device="cuda").bfloat16()
    k, v = row[:, :, :G], row[:, :, G:]
    pool = torch.zeros(330, 2, G, size, hd, dtype=torch.bfloat16, device="cuda")
    kp, vp = pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2)
    table = torch.randperm(330, generator=g, device="cuda").int().view(1, -1)
    f = dc.dynconv_rope_freqs(hd)
    starts = torch.tensor([37], dtype=torch.int32, device="cuda")
    dc.dynconv_attn_paged_store(k, v, kp, vp, table, starts=starts, freqs=f)
    pos = 37 + torch.arange(T, dtype=torch.int32, device="cuda")
    want = dc.dynconv_rope(k, f, positions=pos.view(1, T))
    rows = table[0].long()[pos.long() // size] * size + pos.long() % size
    torch.cuda.synchronize()
    assert torch.equal(kp.reshape(-1, G, hd)[rows], want[0]) and torch.equal(vp.reshape(-1, G, hd)[rows], v[0])
    assert int((kp.reshape(-1, G * hd).abs().sum(1) != 0).sum()) == T


# --- as they are used together ---------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(None, 0), (24, 3)])
def test_prompt_then_steps_follow_the_whole_row(window, sinks, dtype):
    """Ragged prompts attended to and stored, then tokens one at a time, against the whole rows at once."""
    _note(f"[paged] prompt and steps window {window} {dtype}")
    H, G, hd, size, more = 8, 2, 64, 8, 30
    prompts = [40, 1, 75]
    ends = [n + more for n in prompts]
    cu = [0] + [sum(ends[:i + 1]) for i in range(3)]
    g = torch.Generator(device="cuda").manual_seed(11)
    f = dc.dynconv_rope_freqs(hd)
    row = torch.randn(1, cu[-1], H + 2 * G, hd, generator=g, device="cuda").to(au.DTYPES[dtype])
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    qk = dc.dynconv_rope(row[:, :, :H + G], f, cu_seqlens=c)
    whole = (qk[:, :, :H], qk[:, :, H:], row[:, :, H + G:])
    want = (dc.dynconv_attn_fwd(*whole, cu_seqlens=c) if window is None else
            dc.dynconv_attn_window_fwd(*whole, window, sinks=sinks, cu_seqlens=c))[0]
    table = torch.randperm(60, generator=g, device="cuda")[:45].int().view(3, 15)
    kp, vp = (torch.full((60, size, G, hd), math.nan, dtype=row.dtype, device="cuda") for _ in range(2))
    # the prompts as a padded batch
    padded = torch.full((3, 80, H + 2 * G, hd), math.nan, dtype=row.dtype, device="cuda")
    for b, n in enumerate(prompts):
        padded[b, :n] = row[0, cu[b]:cu[b] + n]
    n = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    dc.dynconv_attn_paged_store(padded[:, :, H:H + G], padded[:, :, H + G:], kp, vp, table, counts=n, freqs=f)
    # p of the whole-row call is rounded to bf16, the step's and the outputs' own roundings beside it
    tol = 3 * 2.0 ** -8 if dtype == "bf16" else 1e-5
    for t in range(more):
        new = torch.stack([row[0, cu[b] + prompts[b] + t] for b in range(3)])
        o = dc.dynconv_attn_paged_decode(new[:, :H], new[:, H:H + G], new[:, H + G:], kp, vp, table, n, window=window,
                                         sinks=sinks, freqs=f)
        for b in range(3):
            assert au.rel(o[b], want[cu[b] + prompts[b] + t].double()) <= tol, (t, b)
        n += 1


def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "qkv_attention.py")
    spec = importlib.util.spec_from_file_location("qkv_attention", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def test_the_example_serves_from_pages():
    """The example's ragged prompts and steps: within the roundings of the two ways (p of the whole-row call, the keys and
    the outputs, 2^-8 each, of values that sum to the largest output), in fewer pages than the whole rows have."""
    _note("[paged] example")
    ex = _example()
    off, size, pages = ex.serve()
    assert math.isfinite(off) and off <= 4 * 2.0 ** -7 * size
    assert pages < 3 * 12
    assert all(math.isfinite(x) for x in ex.train(steps=2, window=40, sinks=2))


def test_the_examples_gradients_through_a_window():
    """The layer in fp32: the loss <o, w> along each parameter's gradient, against fourth-order differences.  A step of 1e-4
    of the parameter's norm that way moves the loss by about 1e-4 sqrt(8192 parameters) = 1e-2 of its spread: the
    differences' own error is (1e-2)^4, the loss' roundings (2^-20 of an output, at random) 1.5 * 2^-20 / 1e-2 = 1.4e-4."""
    _note("[paged] example's gradients")
    layer = _example().Layer(32, n_heads=4, n_kv_heads=2, head_dim=32, dtype=torch.float32, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    h = torch.randn(1, 130, 32, generator=g, device="cuda")
    w = torch.randn(1, 130, 4, 32, generator=g, device="cuda").double()
    cu = torch.tensor([0, 50, 130], dtype=torch.int32, device="cuda")

    def loss():
        return (layer.train(h, cu, 24, 2).double() * w).sum()

    loss().backward()
    for name in ("Wp", "W", "w0"):
        p = getattr(layer, name)
        start, grad = p.detach().clone(), p.grad
        u = grad * (1e-4 * start.norm() / grad.norm())

        def along(n):
            with torch.no_grad():
                p.copy_(start + n * u)
                return loss().item()

        diff = (8 * (along(1) - along(-1)) - (along(2) - along(-2))) / 12
        along(0)
        want = (grad.double() * u.double()).sum().item()
        assert abs(diff - want) <= 1e-3 * want, (name, diff, want)


def test_graph_replay():
    """Storing and steps in one graph whose lengths move on, with the eager calls between its replays; two graphs with one
    workspace, one after the other."""
    _note("[paged] graph")
    B, H, G, hd, size, per_seq = 3, 8, 2, 64, 16, 250
    lengths = [1000, 37, -1]
    kp, vp, table = _cache(lengths, per_seq, size, G, hd, "bf16", 21)
    for b in range(2):  # pages for what follows
        free = [i for i in range(kp.shape[0]) if i not in table[:, :].flatten().tolist()]
        table[b, lengths[b] // size + 1] = free[0] if free else -1
    q, k, v = (t.contiguous() for t in _new(B, H, G, hd, "bf16", 22))
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    f = dc.dynconv_rope_freqs(hd)
    pages = dc._pack_pages(kp, vp, table, B, G, hd, kp.dtype, 0)
    a = dc._pack_attn(B, 1, H, G, hd, kp.dtype, 0, None, None)
    ws = torch.empty(dc.lib().dynconv_attn_paged_decode_workspace_bytes(a, None, pages), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0

    def step(kp, vp, n, w, **kw):
        o = dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, n, window=w, sinks=0 if w is None else 2, freqs=f, **kw)
        return o

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(kp.clone(), vp.clone(), n, None)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for w in (None, 1100):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(kp, vp, n, w, workspace=ws))
            n.add_(1)
        graphs.append(graph)
    n.copy_(torch.tensor(lengths, dtype=torch.int32))
    k2, v2, n2 = kp.clone(), vp.clone(), n.clone()
    for r in range(6):
        for t, x in zip((q, k, v), _new(B, H, G, hd, "bf16", 30 + r)):
            t.copy_(x)
        graphs[r % 2].replay()
        torch.cuda.synchronize()
        want = step(k2, v2, n2, (None, 1100)[r % 2])
        n2 += 1
        torch.cuda.synchronize()
        assert torch.equal(outs[r % 2], want) and torch.equal(_bits(kp), _bits(k2)) and torch.equal(n, n2), r


def test_two_streams_and_a_named_one():
    _note("[paged] streams")
    lengths = [2500, 100, 900]
    kp, vp, table = _cache(lengths, 200, 16, 2, 128, "bf16", 31)
    q, k, v = _new(3, 8, 2, 128, "bf16", 32)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want = dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        out = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                out.append(dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, n))
        out.append(dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, n, stream=streams[0]))
        dc.dynconv_attn_paged_store(k[:, None], v[:, None], kp, vp, table, starts=n, stream=streams[0])
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pools_past_4_gib(dtype):
    """Pages at the far end of pools of 5 GiB, split over the cache and not."""
    _note(f"[paged] large pools {dtype}")
    G, hd, size, H = 8, 128, 32, 8
    eb = 2 if dtype == "bf16" else 4
    n_pages = 5 * 2 ** 30 // (size * G * hd * eb)
    dt = au.DTYPES[dtype]
    kp, vp = (torch.empty(n_pages, size, G, hd, dtype=dt, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(41)
    for per_seq, lengths in ((2, [40, 63]), (60, [1900, 10])):
        table = torch.stack([torch.arange(per_seq), torch.arange(n_pages - per_seq, n_pages)]).int().cuda()
        table[0] = table[0].flip(0)
        table[0, 0] = n_pages - per_seq - 1
        T = max(lengths)
        prompt = torch.randn(2, T, 2 * G, hd, generator=g, device="cuda").to(dt)
        n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        dc.dynconv_attn_paged_store(prompt[:, :, :G], prompt[:, :, G:], kp, vp, table, counts=n)
        q, k, v = _new(2, H, G, hd, dtype, 42)
        o = dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, n)
        torch.cuda.synchronize()
        for b, m in enumerate(lengths):
            keys = torch.cat((prompt[b, :m, :G], k[b:b + 1])).double()
            values = torch.cat((prompt[b, :m, G:], v[b:b + 1])).double()
            for h in range(H):
                p = (keys[:, h] @ q[b, h].double() * hd ** -0.5).softmax(0)
                assert au.rel(o[b, h], p @ values[:, h]) <= TOL[dtype]
            page = int(table[b, m // size])
            assert torch.equal(kp[page, m % size], k[b]) and torch.equal(vp[page, m % size], v[b])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths,per_seq", [([40] * 3, 8), ([40] * 40, 250), ([40, 4000, 3, 0], 300)], ids=["whole", "flat", "joined"])
def test_infinite_values_without_weight(lengths, per_seq, dtype):
    """Scores that are all -infinity give zeros also where the values are infinite or NaN: taken whole, as one of several sequences
    of a block, and joined from several blocks."""
    _note(f"[paged] infinite values, scores all -infinity, {len(lengths)} {per_seq} {dtype}")
    B, size = len(lengths), 16
    kp, vp, table = _cache(lengths, per_seq, size, 2, 64, dtype, 51)
    q, k, v = (t.clone() for t in _new(B, 4, 2, 64, dtype, 52))
    q[:, :2, 3] = 1.0
    k[:, 0, 3] = -math.inf
    kp[:, :, 0, 3] = -math.inf
    v[:, 0, 7] = math.inf
    vp[:, 3, 0, 11], vp[:, 5, 0, 12] = -math.inf, math.nan
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ref = wu.paged_decode(q, k, v, kp, vp, table, n)
    o = dc.dynconv_attn_paged_decode(q, k, v, kp, vp, table, n)
    torch.cuda.synchronize()
    assert bool((o[:, :2] == 0).all()) and au.rel(o, ref) <= TOL[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,G", [(128, 8), (272, 16)], ids=["one column block", "two"])
def test_eight_units_of_sixteen_heads_side_by_side(H, G, dtype):
    """The flat launch at the most LDS it takes: eight waves of 16 query heads of 128 (two column blocks: four sets of them)."""
    _note(f"[paged] {H} + {G} heads of 128 {dtype}")
    _step([3300, 70, -1, 5000], 320, 16, H, G, 128, dtype)
    _step([3300, 70, -1, 5000], 320, 16, H, G, 128, dtype, 4000, 5)
