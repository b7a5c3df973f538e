"""Argument checks of the windowed attention calls that need no GPU: every refusal happens on the host, before
anything is enqueued (fake, never dereferenced device addresses), and workspace sizes."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import input_dependent_depthwise_amd as dc
from input_dependent_depthwise_amd import Attn, View, Window

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
    a = dict(B=2, T=1000, n_heads=8, n_kv_heads=2, head_dim=64, dtype=dc.DYNCONV_BF16, scale=0.0, reserved=0,
             cu_seqlens=None, n_seqs=0)
    a.update(kw)
    return Attn(*a.values())


def view(i, heads, hd=64, T=1000):
    return View(addr(i), T * heads * hd, heads * hd, hd)


def fwd(L, a=None, w=Window(100, 4), q=None, k=None, v=None, o=None, lse=addr(9)):
    return L.dynconv_attn_window_fwd(ref(a or attn()), ref(w), ref(q or view(0, 8)), ref(k or view(1, 2)),
                                     ref(v or view(2, 2)), ref(o or view(3, 8)), lse, None)


def need(L, a=None, w=Window(100, 4)):
    return L.dynconv_attn_window_bwd_workspace_bytes(ref(a or attn()), ref(w))


def bwd(L, a=None, w=Window(100, 4), dq=None, dk=None, dv=None, ws=addr(15), nbytes=None, lse=addr(9), d_o=None):
    a = a or attn()
    return L.dynconv_attn_window_bwd(ref(a), ref(w), ref(view(0, 8)), ref(view(1, 2)), ref(view(2, 2)), ref(view(3, 8)),
                                     lse, ref(d_o or view(4, 8)), ref(dq or view(5, 8)), ref(dk or view(6, 2)),
                                     ref(dv or view(7, 2)), ws, need(L, a, w) if nbytes is None else nbytes, None)


def test_struct_size_matches_the_packing():
    assert len(dc._WINDOW(1, 2)) == ctypes.sizeof(Window)


@pytest.mark.parametrize("w,want", [(None, NULL), (Window(0, 4), SHAPE), (Window(-1, 0), SHAPE), (Window(5, -1), SHAPE),
                                    (Window(5, 129), LIMIT), (Window(2000, 129), LIMIT)])
def test_windows(L, w, want):
    assert fwd(L, w=w) == want and bwd(L, w=w, nbytes=1 << 40) == want and need(L, w=w) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=7), DTYPE),
    (dict(n_kv_heads=3), SHAPE),
    (dict(head_dim=60), SHAPE),
    (dict(head_dim=136), LIMIT),
    (dict(scale=-1.0), SHAPE),
    (dict(scale=2.0 ** -121), SHAPE),
    (dict(T=1 << 31), LIMIT),
    (dict(cu_seqlens=addr(20), n_seqs=3), SHAPE),               # B is 2
    (dict(B=1, cu_seqlens=addr(20) + 2, n_seqs=3), ALIGN),
    (dict(B=0), OK),
    (dict(T=0), OK),
])
def test_sizes(L, kw, want):
    assert fwd(L, attn(**kw)) == want
    assert bwd(L, attn(**kw), nbytes=1 << 40) == want


def test_pointers_and_overlaps(L):
    a = attn()
    assert L.dynconv_attn_window_fwd(None, ref(Window(5, 0)), *[ref(view(i, 8)) for i in range(4)], None, None) == NULL
    assert fwd(L, v=View(None, 1, 1, 1)) == NULL
    assert fwd(L, q=View(addr(0) + 8, 512000, 512, 64)) == ALIGN
    assert fwd(L, o=view(0, 8)) == ALIAS
    assert fwd(L, lse=addr(3)) == ALIAS
    assert bwd(L, lse=None) == NULL
    assert bwd(L, ws=None) == WORKSPACE
    assert bwd(L, nbytes=need(L) - 1) == WORKSPACE
    assert bwd(L, ws=addr(15) + 8) == ALIGN
    assert bwd(L, ws=addr(5)) == ALIAS
    assert bwd(L, dk=view(7, 2), dv=view(7, 2)) == ALIAS
    # the sinks' part is the end of the workspace
    plain = need(L, w=Window(100, 0))
    assert need(L) > plain and bwd(L, dq=View(addr(15) + plain + 256, 512000, 512, 64)) == ALIAS


def test_workspace_sizes(L):
    a = attn()
    # few tokens: a slot of 128 queries for each batch row and key/value head: dk and dv of each sink, fp32
    assert need(L, a, Window(100, 4)) - need(L, a, Window(100, 0)) == 2 * 2 * 8 * 4 * 2 * 64 * 4
    p = attn(B=1, cu_seqlens=addr(20), n_seqs=3)
    assert need(L, p, Window(100, 4)) - need(L, p, Window(100, 0)) == 1 * 2 * 8 * 4 * 2 * 64 * 4
    # 8 * 512 blocks of 128 queries: slots of 1024 queries, packed one for each document that can end in them (8)
    a = attn(B=1, T=262144)
    assert need(L, a, Window(100, 4)) - need(L, a, Window(100, 0)) == 2 * 256 * 4 * 2 * 64 * 4
    p = attn(B=1, T=262144, cu_seqlens=addr(20), n_seqs=3)
    assert need(L, p, Window(100, 4)) - need(L, p, Window(100, 0)) == 2 * 256 * 8 * 4 * 2 * 64 * 4
    a = attn()
    # no query past the window of the first 128 keys; a window of the whole row is none
    assert need(L, a, Window(900, 4)) == need(L, a, Window(900, 0))
    assert need(L, a, Window(1000, 4)) == L.dynconv_attn_bwd_workspace_bytes(ref(a))


def test_binding_refuses_before_the_call():
    x = torch.zeros(1, 4, 2, 64)
    for window, sinks, error in ((0, 0, ValueError), (-3, 0, ValueError), (4, -1, ValueError), (4, 129, ValueError),
                                 (4.0, 0, TypeError), (None, 0, TypeError), (4, None, TypeError)):
        with pytest.raises(error):
            dc.dynconv_attn_window_fwd(x, x, x, window, sinks=sinks)
        with pytest.raises(error):
            dc.dynconv_attn_window_bwd(x, x, x, x, x, x, window, sinks=sinks)
    with pytest.raises(TypeError):
        dc.dynconv_attn_window_fwd(x, x, x, 4)  # not on the GPU


def test_the_path_refuses_sinks_without_a_window():
    row = torch.zeros(1, 4, 4 * 64)
    with pytest.raises(ValueError, match="sinks need a window"):
        dc.QKVAttnFn.apply(row, 2, 1, None, False, 1.0, None, None, None, 4)
