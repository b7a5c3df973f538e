"""The Q/K/V path as one: QKVAttnFn (rotary, attention, and the backward into one
gradient row) against fp64 autograd of the definition, behind the convolution's
own autograd wrapper, and the example that trains and decodes with it."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import input_dependent_depthwise_amd as dc
from tests import attn_util as au

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "qkv_attention.py")


def _reference(row, H, G, freqs, interleaved, factor, cu, d_o):
    """o and the gradient of the row by torch autograd in fp64."""
    row = row.double().detach().requires_grad_()
    B, T = row.shape[:2]
    x = row.view(B, T, H + 2 * G, -1)
    t = torch.arange(T, device="cuda")
    start = torch.zeros(T, dtype=torch.int64, device="cuda")
    for lo in cu or []:
        start[lo:] = lo
    ang = (t - start).double()[:, None, None] * freqs
    rot = 2 * freqs.numel()
    part = x[:, :, :H + G, :rot]
    pair = part.unflatten(-1, (rot // 2, 2)) if interleaved else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    a, b = pair.unbind(-1)
    out = torch.stack((a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()), -1) * factor
    out = out.flatten(-2) if interleaved else out.transpose(-1, -2).flatten(-2)
    qk = torch.cat((out, x[:, :, :H + G, rot:]), -1)
    q, k, v = qk[:, :, :H], qk[:, :, H:].repeat_interleave(H // G, 2), x[:, :, H + G:].repeat_interleave(H // G, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, k) * q.shape[-1] ** -0.5
    hidden = (t[:, None] < t[None]) | (start[:, None] != start[None])
    o = torch.einsum("bhij,bjhd->bihd", s.masked_fill(hidden, -torch.inf).softmax(-1), v)
    (o * d_o.double()).sum().backward()
    return o.detach(), row.grad


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved,rot,cu", [(False, 64, None), (True, 32, [0, 50, 131]), (False, 64, [0, 131])])
def test_autograd(interleaved, rot, cu, dtype):
    H, G, hd, T = 4, 2, 64, 131
    B = 2 if cu is None else 1
    g = torch.Generator(device="cuda").manual_seed(3)
    row = torch.randn(B, T, (H + 2 * G) * hd, generator=g, device="cuda").to(au.DTYPES[dtype]).requires_grad_()
    d_o = torch.randn(B, T, H, hd, generator=g, device="cuda").to(au.DTYPES[dtype])
    f = dc.dynconv_rope_freqs(rot)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = dc.QKVAttnFn.apply(row, H, G, f, interleaved, 1.1, None, c)
    o.backward(d_o)
    want_o, want = _reference(row, H, G, f, interleaved, 1.1, cu, d_o)
    # bf16: the turned q and k and the gradients before they are turned back are rounded too (2^-8 each)
    tol = au.TOL[dtype] + (3 * 2.0 ** -8 if dtype == "bf16" else 0.0)
    assert au.rel(o, want_o) <= tol
    assert au.rel(row.grad, want) <= tol


def test_behind_the_convolution():
    """Gradients reach the convolution's inputs and weights through both wrappers."""
    H, G, hd, B, T, d = 4, 1, 32, 2, 50, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    D = (H + 2 * G) * hd
    h, x = (torch.randn(B, T, n, generator=g, device="cuda").requires_grad_() for n in (d, D))
    W = (0.1 * torch.randn(d, (H + 2 * G) * 4, generator=g, device="cuda")).requires_grad_()
    f = dc.dynconv_rope_freqs(hd)
    row = dc.DynConvFn.apply(h, x, W, None, None, None, 4, H + 2 * G)
    row.retain_grad()
    o = dc.QKVAttnFn.apply(row, H, G, f)
    d_o = torch.randn(o.shape, generator=g, device="cuda")
    o.backward(d_o)
    want_o, want = _reference(row, H, G, f, False, 1.0, None, d_o)
    assert au.rel(o, want_o) <= au.TOL["fp32"] and au.rel(row.grad, want) <= au.TOL["fp32"]
    assert all(t.grad is not None and bool(torch.isfinite(t.grad).all()) for t in (h, x, W))


def test_example():
    spec = importlib.util.spec_from_file_location("qkv_attention", EXAMPLE)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses = ex.train()
    assert losses[-1] < losses[0], losses
    off, size = ex.decode()
    # two bf16 paths through projection, convolution, rotary and attention: some roundings of 2^-8 each
    assert off <= 8 * 2.0 ** -8 * size, (off, size)


@pytest.mark.parametrize("B,T", [(2, 0), (0, 7)])
def test_autograd_of_no_tokens(B, T):
    print(f"[path] {B} rows of {T} tokens", flush=True)
    freqs = dc.dynconv_rope_freqs(32, 10000.0).cuda()
    row = torch.zeros(B, T, 4 * 32, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    o = dc.QKVAttnFn.apply(row, 2, 1, freqs)
    assert o.shape == (B, T, 2, 32)
    o.float().sum().backward()
    assert row.grad.shape == row.shape


def test_autograd_of_a_part_of_a_wider_row_and_a_broadcast_gradient():
    print("[path] part of a wider row", flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    freqs = dc.dynconv_rope_freqs(32, 10000.0).cuda()
    wide = torch.randn(2, 77, 200, generator=g, device="cuda").bfloat16()
    part, plain = wide[:, :, 40:168].requires_grad_(), wide[:, :, 40:168].contiguous().requires_grad_()
    for row in (part, plain):
        dc.QKVAttnFn.apply(row, 2, 1, freqs).sum().backward()  # d_o has strides of 0
    assert torch.equal(part.grad, plain.grad)
    with pytest.raises(ValueError):
        dc.QKVAttnFn.apply(plain, 2, 1, freqs, False, 1.0, 0.0)


def test_second_derivatives_are_refused():
    """The gradients carry no history of their own: differentiating them raises instead of leaving this part out."""
    print("[path] second derivatives", flush=True)
    g = torch.Generator(device="cuda").manual_seed(6)
    freqs = dc.dynconv_rope_freqs(32, 10000.0)
    row = torch.randn(1, 20, 4 * 32, generator=g, device="cuda").requires_grad_()
    h, x = (torch.randn(1, 20, 32, generator=g, device="cuda").requires_grad_() for _ in range(2))
    w0 = torch.randn(32, 4, generator=g, device="cuda").requires_grad_()
    for part, leaves in ((dc.QKVAttnFn.apply(row, 2, 1, freqs), [row]),
                         (dc.DynConvFn.apply(h, x, None, None, None, w0, 4, 0), [x, w0])):
        # another part of the loss has a second derivative
        loss = part.square().sum() + sum(t.pow(3).sum() for t in leaves)
        first = torch.autograd.grad(loss, leaves, create_graph=True)
        assert all(bool(torch.isfinite(t).all()) for t in first)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            sum(t.square().sum() for t in first).backward()


def test_a_workspace_of_the_callers():
    """One that is on the GPU and whole is used, others are refused before the call."""
    print("[path] workspace", flush=True)
    g = torch.Generator(device="cuda").manual_seed(8)
    q, k, v, d_o = (torch.randn(1, 300, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(4))
    o, lse = dc.dynconv_attn_fwd(q, k, v, want_lse=True)
    want = dc.dynconv_attn_bwd(q, k, v, o, lse, d_o)
    room = torch.empty(1 << 20, device="cuda")
    got = dc.dynconv_attn_bwd(q, k, v, o, lse, d_o, workspace=room)
    assert all(torch.equal(got[n], want[n]) for n in want)
    cache = torch.zeros(1, 4000, 2, 64, dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (torch.empty(1 << 20), room[::2]):
        with pytest.raises(TypeError, match="workspace"):
            dc.dynconv_attn_bwd(q, k, v, o, lse, d_o, workspace=bad)
        with pytest.raises(TypeError, match="workspace"):
            dc.dynconv_attn_decode(q[:, 0], k[:, 0], v[:, 0], cache, cache.clone(), n, workspace=bad)
