"""Argument checks of the calls on a cache kept in pages that need no GPU: every refusal happens on the host, before
anything is enqueued (fake, never dereferenced device addresses), workspace sizes, and the binding."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import input_dependent_depthwise_amd as dc
from input_dependent_depthwise_amd import Attn, Pages, Rotary, View, Window
from tests.test_attn_abi_cpu import OnGPU

OK, NULL, SHAPE, DTYPE, ALIGN, ALIAS, WORKSPACE, LIMIT = 0, -1, -2, -4, -5, -6, -7, -9
MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dc.LIB_PATH):
        from input_dependent_depthwise_amd import build
        build.build()
    return dc.lib()


def addr(i):
    return (1 << 40) + i * 64 * MB


def ref(x):
    return None if x is None else ctypes.byref(x)


def attn(**kw):
    a = dict(B=2, T=1, n_heads=8, n_kv_heads=2, head_dim=64, dtype=dc.DYNCONV_BF16, scale=0.0, reserved=0,
             cu_seqlens=None, n_seqs=0)
    a.update(kw)
    return Attn(*a.values())


def view(i, heads, hd=64, T=1):
    return View(addr(i), T * heads * hd, heads * hd, hd)


def pages(**kw):
    p = dict(k=View(addr(5), 16 * 128, 128, 64), v=View(addr(6), 16 * 128, 128, 64), table=addr(7), table_row=200,
             n_pages=400, pages_per_seq=200, page_size=16, reserved=0)
    p.update(kw)
    return Pages(*p.values())


ROT = Rotary(64, 0, 0, 1.0, addr(8))


def step(L, a=None, w=None, r=None, q=None, k=None, v=None, p=None, n=addr(9), o=None, ws=addr(10), nbytes=1 << 26):
    return L.dynconv_attn_paged_decode(ref(a or attn()), ref(w), ref(r), ref(q or view(0, 8)), ref(k or view(1, 2)),
                                       ref(v or view(2, 2)), ref(p or pages()), n, ref(o or view(3, 8)), ws, nbytes, None)


def store(L, a=None, r=None, k=None, v=None, p=None, starts=addr(9), counts=None):
    return L.dynconv_attn_paged_store(ref(a or attn(T=30)), ref(r), ref(k or view(1, 2, T=30)), ref(v or view(2, 2, T=30)),
                                      ref(p or pages()), starts, counts, None)


def test_struct_size_matches_the_packing():
    raw = dc._PAGES(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 0)
    assert len(raw) == ctypes.sizeof(Pages)
    p = Pages.from_buffer_copy(raw)
    assert (p.k.data, p.k.head, p.v.data, p.v.head, p.table, p.table_row, p.n_pages, p.pages_per_seq, p.page_size) == (
        1, 4, 5, 8, 9, 10, 11, 12, 13)


@pytest.mark.parametrize("kw,want", [
    (dict(n_pages=0), SHAPE),
    (dict(pages_per_seq=0), SHAPE),
    (dict(page_size=0), SHAPE),
    (dict(page_size=-16), SHAPE),
    (dict(n_pages=1 << 31), LIMIT),
    (dict(pages_per_seq=1 << 28), LIMIT),                        # 2^32 positions
    (dict(k=View(None, 2048, 128, 64)), NULL),
    (dict(v=View(addr(6) + 8, 2048, 128, 64)), ALIGN),
    (dict(v=View(addr(6), 2044, 128, 64)), ALIGN),
    (dict(table=None), NULL),
    (dict(table=addr(7) + 2), ALIGN),
    (dict(table_row=-1), SHAPE),
    (dict(table_row=1 << 60), LIMIT),
    (dict(v=View(addr(5), 2048, 128, 64)), ALIAS),               # keys and values in one place
    (dict(k=View(addr(5), 2048, 64, 64)), ALIAS),                # rows that overlap
    (dict(k=View(addr(5), 1024, 128, 64)), ALIAS),               # pages that overlap
    (dict(table=addr(5) + 400), ALIAS),
])
def test_pages(L, kw, want):
    assert step(L, p=pages(**kw)) == want
    assert store(L, p=pages(**kw)) == want
    assert L.dynconv_attn_paged_decode_workspace_bytes(ref(attn()), None, ref(pages(**kw))) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=7), DTYPE),
    (dict(n_kv_heads=3), SHAPE),
    (dict(head_dim=60), SHAPE),
    (dict(head_dim=136), LIMIT),
    (dict(scale=-1.0), SHAPE),
    (dict(T=2), SHAPE),
    (dict(B=1, cu_seqlens=addr(20), n_seqs=1), SHAPE),
    (dict(B=65536), LIMIT),
    (dict(B=65535, n_heads=1024, n_kv_heads=1024), LIMIT),
    (dict(B=0), OK),
])
def test_step_sizes(L, kw, want):
    assert step(L, attn(**kw)) == want


def test_step_pointers_and_overlaps(L):
    a, p = attn(), pages()
    need = L.dynconv_attn_paged_decode_workspace_bytes(ref(a), None, ref(p))
    assert need > 0
    assert step(L, w=Window(0, 1)) == SHAPE and step(L, w=Window(4, 129)) == LIMIT
    assert L.dynconv_attn_paged_decode(ref(a), None, None, ref(view(0, 8)), ref(view(1, 2)), ref(view(2, 2)), None, addr(9),
                                       ref(view(3, 8)), addr(10), 1 << 26, None) == NULL
    assert step(L, n=None) == NULL
    assert step(L, n=addr(9) + 1) == ALIGN
    assert step(L, q=View(addr(0) + 2, 512, 512, 64)) == ALIGN
    assert step(L, r=Rotary(64, 0, 1, 1.0, addr(8))) == SHAPE
    assert step(L, r=Rotary(66, 0, 0, 1.0, addr(8))) == SHAPE
    assert step(L, r=Rotary(64, 0, 0, 1.0, None)) == NULL
    assert step(L, ws=None) == WORKSPACE and step(L, nbytes=need - 1) == WORKSPACE
    assert step(L, ws=addr(10) + 4) == ALIGN
    assert step(L, o=view(0, 8)) == ALIAS
    assert step(L, o=view(5, 8)) == ALIAS
    assert step(L, k=view(6, 2)) == ALIAS
    assert step(L, n=addr(5) + 4096) == ALIAS
    assert step(L, ws=addr(6)) == ALIAS
    assert step(L, ws=addr(3)) == ALIAS
    assert step(L, ws=addr(7) - need + 16) == ALIAS
    assert step(L, r=Rotary(64, 0, 0, 1.0, addr(10))) == ALIAS


def test_store_arguments(L):
    assert store(L, r=Rotary(64, 0, 1, 1.0, addr(8))) == SHAPE
    assert store(L, attn(B=1, T=30, cu_seqlens=addr(20), n_seqs=2), counts=addr(21)) == SHAPE
    assert store(L, attn(T=30, cu_seqlens=addr(20), n_seqs=2)) == SHAPE                 # B is 2
    assert store(L, starts=addr(9) + 2) == ALIGN
    assert store(L, counts=addr(9) + 1) == ALIGN
    assert store(L, k=View(None, 1, 1, 1)) == NULL
    assert store(L, k=view(5, 2, T=30)) == ALIAS
    assert store(L, starts=addr(6) + 64) == ALIAS
    assert store(L, counts=addr(5)) == ALIAS
    assert store(L, r=Rotary(64, 0, 0, 1.0, addr(6))) == ALIAS
    assert store(L, attn(B=1 << 20, T=1 << 11)) == LIMIT
    assert store(L, attn(T=0)) == OK and store(L, attn(B=0, T=30)) == OK
    assert store(L, attn(dtype=5, T=30)) == DTYPE


def test_workspace_sizes(L):
    need = lambda a, w, p: L.dynconv_attn_paged_decode_workspace_bytes(ref(a), ref(w), ref(p))  # noqa: E731
    a = attn()
    assert need(a, None, pages(pages_per_seq=60)) == 0              # 960 tokens: a block reads them
    assert need(a, Window(500, 4), pages()) == 0                    # as does a window of 500
    full = need(a, None, pages())
    assert full > 0 and need(a, Window(3200, 4), pages()) == full   # a window of all positions is none
    assert need(attn(B=1025), None, pages(table_row=200)) == 0      # enough sequences for the chip


def test_binding_refuses_before_the_call():
    bf, i32 = torch.bfloat16, torch.int32
    q, k = OnGPU(1, (2, 8, 64)), OnGPU(1, (2, 2, 64))
    pool, table, n = OnGPU(1, (40, 16, 2, 64)), OnGPU(1, (2, 20), i32), OnGPU(1, (2,), i32)
    call = dc.dynconv_attn_paged_decode
    good = dict(q=q, k=k, v=k, k_pages=pool, v_pages=pool, page_table=table, lengths=n, o=q)
    for kw, error in ((dict(sinks=2), ValueError), (dict(window=0), ValueError), (dict(window=4, sinks=200), ValueError),
                      (dict(v_pages=OnGPU(1, (40, 8, 2, 64))), ValueError), (dict(k_pages=OnGPU(1, (40, 16, 64))), ValueError),
                      (dict(v_pages=OnGPU(1, (40, 16, 2, 64), torch.float32)), TypeError),
                      (dict(page_table=OnGPU(1, (3, 20), i32)), TypeError), (dict(page_table=OnGPU(1, (2, 20), bf)), TypeError),
                      (dict(page_table=OnGPU(0, (2, 20), i32)), ValueError), (dict(v_pages=OnGPU(0, (40, 16, 2, 64))), ValueError),
                      (dict(lengths=OnGPU(1, (3,), i32)), TypeError), (dict(lengths=OnGPU(0, (2,), i32)), ValueError),
                      (dict(scale=0.0), ValueError), (dict(k=OnGPU(1, (3, 2, 64))), ValueError)):
        with pytest.raises(error):
            call(**{**good, **kw})
    x = OnGPU(1, (2, 30, 2, 64))
    good = dict(k=x, v=x, k_pages=pool, v_pages=pool, page_table=table)
    for kw, error in ((dict(starts=OnGPU(1, (3,), i32)), TypeError), (dict(counts=OnGPU(1, (2,), bf)), TypeError),
                      (dict(counts=OnGPU(0, (2,), i32)), ValueError), (dict(page_table=OnGPU(1, (1, 20), i32)), TypeError),
                      (dict(v=OnGPU(1, (2, 31, 2, 64))), ValueError), (dict(v=OnGPU(0, (2, 30, 2, 64))), ValueError),
                      (dict(cu_seqlens=OnGPU(1, (3,), i32), counts=n), ValueError)):
        with pytest.raises(error):
            dc.dynconv_attn_paged_store(**{**good, **kw})


def test_launches_go_to_the_tensors_gpu(monkeypatch):
    """A launch goes to the current device: it is the tensors' for the time of the call, with its own current stream."""
    import contextlib
    seen, current = [], [0]

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)

    class Lib:
        def dynconv_attn_paged_store(self, *args):
            seen.append((current[0], args[-1]))
            return 0

        dynconv_attn_paged_decode = dynconv_attn_window_fwd = dynconv_attn_paged_store

        def dynconv_attn_paged_decode_workspace_bytes(self, *args):
            return 0

    monkeypatch.setattr(dc, "lib", Lib)
    i32 = torch.int32
    for i in (0, 1, 0):
        q, k = OnGPU(i, (2, 8, 64)), OnGPU(i, (2, 2, 64))
        pool, table, n, x = OnGPU(i, (40, 16, 2, 64)), OnGPU(i, (2, 20), i32), OnGPU(i, (2,), i32), OnGPU(i, (2, 30, 2, 64))
        dc.dynconv_attn_paged_decode(q, k, k, pool, pool, table, n, o=q)
        dc.dynconv_attn_paged_store(x, x, pool, pool, table)
        dc.dynconv_attn_window_fwd(x, x, x, 4, o=x)
    assert seen == [(i, 1000 + i) for i in (0, 0, 0, 1, 1, 1, 0, 0, 0)] and current == [0]


@pytest.mark.parametrize("size,most", [((1 << 31) - 4097, 1), (1 << 30, 1), (300_000_000, 7), (1000, 2147479), (3, 715826517),
                                       (1, (1 << 31) - 4097)])
def test_positions_up_to_the_limit(L, size, most):
    """page_size * pages_per_seq: the last product below 2^31 - 4096 is taken (what is refused then is the lengths' missing
    address), one page more is not."""
    assert size * most < (1 << 31) - 4096 <= size * (most + 1)
    side_by_side = dict(k=View(addr(5), 0, 256, 64), v=View(addr(5) + 256, 0, 256, 64), table=addr(-200), n_pages=1, page_size=size)
    assert step(L, attn(B=1), p=pages(pages_per_seq=most, table_row=0, **side_by_side), n=None) == NULL
    assert step(L, attn(B=1), p=pages(pages_per_seq=most + 1, table_row=0, **side_by_side), n=None) == LIMIT
    assert store(L, attn(B=1, T=30), p=pages(pages_per_seq=most, table_row=0, **side_by_side), k=View(None, 1, 1, 1)) == NULL
    assert store(L, attn(B=1, T=30), p=pages(pages_per_seq=most + 1, table_row=0, **side_by_side), k=View(None, 1, 1, 1)) == LIMIT
