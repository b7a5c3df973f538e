"""Argument checks of the rotary and attention calls that need no GPU: every
refusal happens on the host, before anything is enqueued (fake, never
dereferenced device addresses), workspace sizes, and the host-side frequencies."""
from __future__ import annotations

import ctypes
import math
import os

import pytest

import input_dependent_depthwise_amd as dc
from input_dependent_depthwise_amd import Attn, Rotary, View

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
    a = dict(B=2, T=100, n_heads=8, n_kv_heads=2, head_dim=64, dtype=dc.DYNCONV_BF16, scale=0.0, reserved=0,
             cu_seqlens=None, n_seqs=0)
    a.update(kw)
    return Attn(*a.values())


def view(i, heads, hd=64, T=100):
    return View(addr(i), T * heads * hd, heads * hd, hd)


def fwd(L, a=None, q=None, k=None, v=None, o=None, lse=addr(9)):
    a = a or attn()
    return L.dynconv_attn_fwd(ref(a), ref(q or view(0, 8)), ref(k or view(1, 2)), ref(v or view(2, 2)),
                              ref(o or view(3, 8)), lse, None)


def test_struct_sizes_match_the_packing():
    assert len(dc._VIEW(1, 2, 3, 4)) == ctypes.sizeof(View)
    assert len(dc._ATTN(1, 2, 3, 4, 5, 6, 0.5, 0, 7, 8)) == ctypes.sizeof(Attn)
    assert len(dc._ROTARY(1, 2, 3, 0.5, 4)) == ctypes.sizeof(Rotary)
    a, b = Attn.from_buffer_copy(dc._ATTN(1, 2, 3, 4, 5, 6, 0.5, 0, 7, 8)), Rotary.from_buffer_copy(dc._ROTARY(1, 2, 3, 0.5, 4))
    assert (a.B, a.T, a.n_heads, a.n_kv_heads, a.head_dim, a.dtype, a.scale, a.cu_seqlens, a.n_seqs) == (1, 2, 3, 4, 5, 6, 0.5, 7, 8)
    assert (b.rot_dim, b.interleaved, b.inverse, b.factor, b.freqs) == (1, 2, 3, 0.5, 4)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=7), DTYPE),
    (dict(B=-1), SHAPE),
    (dict(n_heads=0), SHAPE),
    (dict(n_kv_heads=0), SHAPE),
    (dict(n_kv_heads=3), SHAPE),
    (dict(head_dim=0), SHAPE),
    (dict(head_dim=60), SHAPE),
    (dict(head_dim=136), LIMIT),
    (dict(dtype=dc.DYNCONV_FP32, head_dim=66), SHAPE),
    (dict(scale=-1.0), SHAPE),
    (dict(scale=math.inf), SHAPE),
    (dict(scale=math.nan), SHAPE),
    (dict(T=1 << 31), LIMIT),
    (dict(B=1 << 20, T=1 << 20), LIMIT),
    (dict(cu_seqlens=addr(20), n_seqs=3), SHAPE),               # B is 2
    (dict(B=1, cu_seqlens=addr(20), n_seqs=0), SHAPE),
    (dict(B=1, cu_seqlens=addr(20) + 2, n_seqs=3), ALIGN),
    (dict(B=0), OK),
    (dict(T=0), OK),
])
def test_sizes(L, kw, want):
    assert fwd(L, attn(**kw)) == want


def test_forward_pointers(L):
    a = attn()
    assert L.dynconv_attn_fwd(None, ref(view(0, 8)), ref(view(1, 2)), ref(view(2, 2)), ref(view(3, 8)), None, None) == NULL
    assert L.dynconv_attn_fwd(ref(a), None, ref(view(1, 2)), ref(view(2, 2)), ref(view(3, 8)), None, None) == NULL
    assert fwd(L, v=View(None, 1, 1, 1)) == NULL
    assert fwd(L, q=View(addr(0) + 8, 51200, 512, 64)) == ALIGN
    assert fwd(L, q=View(addr(0), 51200, 516, 64)) == ALIGN
    assert fwd(L, q=View(addr(0), 51200, 512, -64)) == SHAPE
    assert fwd(L, k=View(addr(1), 12800, 1 << 40, 64)) == LIMIT
    assert fwd(L, k=View(addr(1), 12800, 16 * MB, 64)) == LIMIT       # a row of 32 MiB
    assert fwd(L, k=View(addr(1), 1 << 61, 128, 64)) == LIMIT
    assert fwd(L, lse=addr(9) + 2) == ALIGN


def test_forward_overlaps(L):
    assert fwd(L, o=view(0, 8)) == ALIAS
    assert fwd(L, o=View(addr(3), 51200, 512, 0)) == ALIAS            # heads on top of each other
    assert fwd(L, o=View(addr(3), 51200, 256, 64)) == ALIAS           # rows that overlap
    assert fwd(L, lse=addr(3)) == ALIAS
    assert fwd(L, lse=addr(1)) == ALIAS
    # o among the value heads of the row that q, k and v are parts of
    part = lambda first: View(addr(0) + first * 128, 100 * 768, 768, 64)  # noqa: E731
    assert fwd(L, q=part(0), k=part(8), v=part(10), o=part(4)) == ALIAS


def bwd(L, a=None, dq=None, dk=None, dv=None, ws=addr(15), nbytes=None, lse=addr(9), d_o=None):
    a = a or attn()
    n = L.dynconv_attn_bwd_workspace_bytes(ref(a)) if nbytes is None else nbytes
    return L.dynconv_attn_bwd(ref(a), ref(view(0, 8)), ref(view(1, 2)), ref(view(2, 2)), ref(view(3, 8)), lse,
                              ref(d_o or view(4, 8)), ref(dq or view(5, 8)), ref(dk or view(6, 2)), ref(dv or view(7, 2)),
                              ws, n, None)


def test_backward(L):
    need = L.dynconv_attn_bwd_workspace_bytes(ref(attn()))
    assert need >= 2 * 8 * 100 * 4
    assert L.dynconv_attn_bwd_workspace_bytes(ref(attn(head_dim=60))) == 0
    assert L.dynconv_attn_bwd_workspace_bytes(ref(attn(B=0))) == 0
    assert bwd(L, nbytes=need - 1) == WORKSPACE
    assert bwd(L, ws=None) == WORKSPACE
    assert bwd(L, ws=addr(15) + 8) == ALIGN
    assert bwd(L, lse=None) == NULL
    assert bwd(L, dq=view(4, 8)) == ALIAS
    assert bwd(L, dk=view(7, 2)) == ALIAS
    assert bwd(L, ws=addr(5)) == ALIAS
    assert bwd(L, attn(B=0)) == OK


def decode(L, a=None, r=None, cap=500, kc=None, vc=None, n=addr(12), o=None, ws=addr(15), nbytes=1 << 24, k=None):
    a = a or attn(T=1)
    return L.dynconv_attn_decode(ref(a), ref(r), ref(view(0, 8, T=1)), ref(k or view(1, 2, T=1)), ref(view(2, 2, T=1)),
                                 ref(kc or view(5, 2, T=cap)), ref(vc or view(6, 2, T=cap)), cap, n,
                                 ref(o or view(3, 8, T=1)), ws, nbytes, None)


def test_decode(L):
    assert decode(L, attn(T=2)) == SHAPE
    assert decode(L, attn(T=1, B=1, cu_seqlens=addr(20), n_seqs=1)) == SHAPE
    assert decode(L, cap=0) == SHAPE
    assert decode(L, cap=1 << 31) == LIMIT
    assert decode(L, attn(T=1, B=70000)) == LIMIT
    assert decode(L, n=None) == NULL
    assert decode(L, n=addr(12) + 1) == ALIGN
    assert decode(L, vc=view(5, 2, T=500)) == ALIAS
    assert decode(L, o=view(5, 8, T=1)) == ALIAS
    assert decode(L, k=view(5, 2, T=1)) == ALIAS                       # the new key inside the cache
    assert decode(L, r=Rotary(64, 0, 0, 1.0, None)) == NULL
    assert decode(L, r=Rotary(63, 0, 0, 1.0, addr(13))) == SHAPE
    assert decode(L, r=Rotary(66, 0, 0, 1.0, addr(13))) == SHAPE
    assert decode(L, r=Rotary(64, 0, 1, 1.0, addr(13))) == SHAPE       # no turning back here
    assert decode(L, r=Rotary(64, 0, 0, 1.0, addr(13) + 4)) == ALIGN
    need = L.dynconv_attn_decode_workspace_bytes(ref(attn(T=1)), 8192)
    assert need > 0 and L.dynconv_attn_decode_workspace_bytes(ref(attn(T=1)), 512) == 0
    assert decode(L, cap=8192, nbytes=need - 1) == WORKSPACE
    assert decode(L, attn(T=1, B=0)) == OK


def rope(L, a=None, r=None, x=None, y=None, pos=None):
    a, r = a or attn(), r or Rotary(64, 0, 0, 1.0, addr(13))
    return L.dynconv_rope(ref(a), ref(r), ref(x or view(0, 8)), pos, ref(y or view(3, 8)), None)


def test_rope(L):
    assert rope(L, attn(dtype=9)) == DTYPE
    assert rope(L, r=Rotary(0, 0, 0, 1.0, addr(13))) == SHAPE
    assert rope(L, r=Rotary(7, 0, 0, 1.0, addr(13))) == SHAPE
    assert rope(L, r=Rotary(66, 0, 0, 1.0, addr(13))) == SHAPE
    assert rope(L, r=Rotary(64, 0, 0, 1.0, None)) == NULL
    assert rope(L, r=Rotary(64, 0, 0, 1.0, addr(13) + 4)) == ALIGN
    assert rope(L, pos=addr(14) + 1) == ALIGN
    assert rope(L, x=View(addr(0) + 1, 51200, 512, 64)) == ALIGN
    assert rope(L, y=View(addr(0) + 2, 51200, 512, 64)) == ALIAS
    assert rope(L, y=View(addr(3), 51200, 0, 64)) == ALIAS
    assert rope(L, y=view(13, 8)) == ALIAS                             # over the frequencies
    assert rope(L, pos=addr(3)) == ALIAS
    assert rope(L, attn(B=0)) == OK
    assert rope(L, attn(B=1 << 20, T=1 << 20)) == LIMIT


def test_frequencies(L):
    out = (ctypes.c_double * 8)()
    f = L.dynconv_rope_freqs
    assert f(16, 10000.0, 1.0, 0.0, 1.0, 32.0, ctypes.addressof(out)) == OK
    assert list(out) == pytest.approx([10000.0 ** (-m / 8) for m in range(8)], rel=1e-14)
    assert f(16, 10000.0, 1.0, 0.0, 1.0, 32.0, None) == NULL
    for bad in ((15, 1e4, 1.0, 0.0, 1.0, 2.0), (0, 1e4, 1.0, 0.0, 1.0, 2.0), (16, 0.0, 1.0, 0.0, 1.0, 2.0),
                (16, 1e4, 0.5, 0.0, 1.0, 2.0), (16, 1e4, 2.0, -1.0, 1.0, 2.0), (16, 1e4, 2.0, 100.0, 2.0, 2.0),
                (16, math.nan, 1.0, 0.0, 1.0, 2.0), (16, 1e4, math.inf, 0.0, 1.0, 2.0)):
        assert f(*bad, ctypes.addressof(out)) == SHAPE, bad


def test_binding_refuses_before_the_call():
    import torch
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(TypeError):  # host tensors
        dc.dynconv_attn_fwd(x, x, x)
    with pytest.raises(TypeError):
        dc.dynconv_rope(x, f)
    with pytest.raises(ValueError):
        dc.dynconv_attn_fwd(x[0], x, x)
    with pytest.raises(TypeError):
        dc.dynconv_attn_fwd(x.half(), x.half(), x.half())
    with pytest.raises(dc.DynConvError):
        dc.dynconv_rope_freqs(5, device="cpu")


def test_more_threads_than_a_launch_takes(L):
    """2^24 blocks of 256 threads: refused before the launch."""
    assert fwd(L, attn(B=1 << 14, T=128 << 7)) == LIMIT
    assert L.dynconv_attn_bwd_workspace_bytes(ref(attn(B=1 << 14, T=128 << 7))) == 0
    row = View(addr(0), 10 << 18, 10, 10)  # five pairs of single elements, a thread for each
    r = Rotary(10, 0, 0, 1.0, 1 << 42)
    assert rope(L, attn(B=1 << 12, T=1 << 18, n_heads=1, head_dim=10), r=r, x=row, y=row) == LIMIT


def test_a_scale_of_zero_is_not_the_default():
    assert dc._scale(None) == 0.0 and dc._scale(0.5) == 0.5
    for s in (0, 0.0, 1e-39):
        with pytest.raises(ValueError):
            dc._scale(s)


def test_scales_too_small_for_the_backward_are_refused(L):
    """lse / scale would pass the largest float (the calls that need it have to agree on it)."""
    small, least = attn(scale=2.0 ** -121), attn(scale=2.0 ** -120)
    assert fwd(L, small) == SHAPE and bwd(L, small, nbytes=1 << 24) == SHAPE
    assert decode(L, attn(T=1, scale=2.0 ** -126)) == SHAPE
    assert L.dynconv_attn_bwd_workspace_bytes(ref(small)) == 0 < L.dynconv_attn_bwd_workspace_bytes(ref(least))
    with pytest.raises(ValueError):
        dc._scale(2.0 ** -121)
    assert dc._scale(2.0 ** -120) == 2.0 ** -120


def test_rotary_tokens_past_2_gib_are_refused(L):
    """Heads and widths whose product passes the kernels' 32-bit counts (65535 heads of 2^19 elements, bf16)."""
    for heads, hd, dtype, want in ((65535, 1 << 19, dc.DYNCONV_BF16, LIMIT), (65535, 1 << 20, dc.DYNCONV_BF16, LIMIT),
                                   (1, 1 << 30, dc.DYNCONV_BF16, LIMIT), (1, 1 << 29, dc.DYNCONV_FP32, LIMIT)):
        x, y = View(addr(0), 0, 0, 0), View(1 << 45, 0, 0, hd)
        for rot in (64, 4096):
            a = attn(B=1, T=1, n_heads=heads, head_dim=hd, dtype=dtype)
            assert rope(L, a, r=Rotary(rot, 0, 0, 1.0, 1 << 44), x=x, y=y) == want, (heads, hd, dtype, rot)


class OnGPU:
    """What the binding asks of a tensor, on a GPU of the given index."""
    is_cuda = True

    def __init__(self, index, shape=(1, 4, 2, 64), dtype=None):
        import torch
        self.index, self.shape = index, torch.Size(shape)
        self.dtype, self.device = dtype or torch.bfloat16, torch.device("cuda", index)

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def data_ptr(self):
        return addr(self.index)

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return True


def test_launches_go_to_the_tensors_gpu(monkeypatch):
    """A launch goes to the current device: it is the tensors' for the time of the call, with its own current stream."""
    import contextlib

    import torch
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
        def dynconv_rope(self, *args):
            seen.append((current[0], args[-1]))
            return 0

        dynconv_attn_fwd = dynconv_rope

    monkeypatch.setattr(dc, "lib", Lib)
    for index in (0, 1, 0):
        x = OnGPU(index)
        dc.dynconv_rope(x, OnGPU(index, (32,), torch.float64), out=x)
    assert seen == [(0, 1000), (1, 1001), (0, 1000)] and current == [0]
    # tensors of several GPUs, and a stream of another one
    x = OnGPU(1)
    for kw in (dict(freqs=OnGPU(0, (32,), torch.float64)), dict(out=OnGPU(0)), dict(positions=OnGPU(0, (1, 4), torch.int32)),
               dict(cu_seqlens=OnGPU(0, (2,), torch.int32))):
        with pytest.raises(ValueError, match="cuda:1"):
            dc.dynconv_rope(x, **{"freqs": OnGPU(1, (32,), torch.float64), "out": x, **kw})
    for q, k, v in ((x, OnGPU(0), x), (x, x, OnGPU(0))):
        with pytest.raises(ValueError, match="cuda:1"):
            dc.dynconv_attn_fwd(q, k, v, o=OnGPU(1))

    class Stream:
        device = torch.device("cuda", 0)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with pytest.raises(ValueError, match="cuda:1"):
        dc.dynconv_rope(x, OnGPU(1, (32,), torch.float64), out=x, stream=Stream())
    assert len(seen) == 3


def test_a_workspace_of_the_callers_is_checked():
    import torch
    dev = torch.device("cuda", 0)
    host, meta = torch.empty(64, dtype=torch.uint8), torch.empty(64, dtype=torch.uint8, device="meta")
    for bad in (host, meta):
        with pytest.raises(TypeError, match="workspace"):
            dc._workspace(16, dev, bad)
    with pytest.raises(TypeError, match="workspace"):
        dc._workspace(16, host.device, host[::2])  # every other byte of a buffer that is not all the caller's
    assert dc._workspace(16, host.device, host) is host
    with pytest.raises(TypeError, match="workspace"):
        dc._workspace(16, OnGPU(1).device, OnGPU(0, (64,), torch.uint8))


@pytest.fixture
def no_gpu():
    """For calls whose checks pass: they go on to the launch, which fails without a GPU (the addresses are made up)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")


def test_views_that_interleave_pass(L, no_gpu):
    """Parts of one buffer that share no element, whichever axis they alternate on: none of them is an overlap."""
    B, T, H, G, hd = 2, 100, 8, 2, 64
    e, N = 2, H + 2 * G

    def bwd_into(dq, dk, dv):
        a = attn()
        return L.dynconv_attn_bwd(ref(a), ref(view(0, 8)), ref(view(1, 2)), ref(view(2, 2)), ref(view(3, 8)), addr(9),
                                  ref(view(4, 8)), ref(dq), ref(dk), ref(dv), addr(15), 1 << 24, None)

    def at(first, batch, row, head):
        return View(addr(5) + first * e, batch, row, head)

    row = N * hd
    good = {
        "parts of a row": [at(f * hd, T * row, row, hd) for f in (0, H, H + G)],
        "parts of a token, tokens outside": [at(f * hd, row, B * row, hd) for f in (0, H, H + G)],
        "head-major parts of a batch row": [at(f * T * hd, N * T * hd, hd, T * hd) for f in (0, H, H + G)],
        "head-major parts, batches inside": [at(f * T * B * hd, T * hd, hd, B * T * hd) for f in (0, H, H + G)],
    }
    for name, views in good.items():
        assert bwd_into(*views) != ALIAS, name
    # a group's key between its queries and its value: [B, T, G, n + 2, hd] with one query head to a group
    one = attn(n_heads=2, n_kv_heads=2)
    group = [at(i * hd, T * 2 * 3 * hd, 2 * 3 * hd, 3 * hd) for i in range(3)]
    ins = [ref(view(i, 2)) for i in range(5)]
    assert L.dynconv_attn_bwd(ref(one), *ins[:4], addr(9), ins[4], *[ref(v) for v in group], addr(15), 1 << 24, None) != ALIAS
    for i in range(3):  # one element further to the left or right is in the neighbour's head
        for by in (-8, 8):
            moved = list(group)
            moved[i] = View(group[i].data + by * e, group[i].batch, group[i].row, group[i].head)
            assert L.dynconv_attn_bwd(ref(one), *ins[:4], addr(9), ins[4], *[ref(v) for v in moved], addr(15), 1 << 24,
                                      None) == ALIAS
    assert bwd_into(at(0, T * row, row, hd), at((H - 1) * hd, T * row, row, hd), at((H + G) * hd, T * row, row, hd)) == ALIAS
    assert bwd_into(at(0, row, B * row, hd), at(H * hd, row, B * row, hd), at((H + G + 1) * hd, row, B * row, hd)) == ALIAS


def test_overlaps_are_found(L, no_gpu):
    """Small views of one buffer with drawn strides: whatever shares an element is refused."""
    import itertools
    import random
    r = random.Random(3)
    B, T, H, hd, e = 2, 3, 2, 8, 2
    a = attn(B=B, T=T, n_heads=H, n_kv_heads=H, head_dim=hd)
    far = [ref(View(addr(i), T * H * hd, H * hd, hd)) for i in range(2)]

    def elements(v):
        return {(v.data - addr(5)) // e + b * v.batch + t * v.row + h * v.head + i
                for b, t, h, i in itertools.product(range(B), range(T), range(H), range(hd))}

    def drawn():
        s = r.choice(list(itertools.permutations((1, 2, 3, 4, 6, 8, 12), 3)) + [(6, 2, 1), (12, 4, 2), (12, 4, 1), (2, 4, 1)])
        return View(addr(5) + 16 * r.randrange(12), *(8 * x for x in s))

    refused = passed = 0
    for i in range(4000):
        v, o = drawn(), drawn()
        if i % 2:  # the same strides, another place
            o = View(o.data, v.batch, v.row, v.head)
        rc = L.dynconv_attn_fwd(ref(a), *far, ref(v), ref(o), None, None)
        shared = bool(elements(v) & elements(o)) or len(elements(o)) < B * T * H * hd
        assert rc == ALIAS or not shared, (v.data, v.batch, v.row, v.head, o.data, o.batch, o.row, o.head)
        refused, passed = refused + (rc == ALIAS), passed + (rc != ALIAS)
    assert refused > 100 and passed > 100
