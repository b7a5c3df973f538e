"""Rotary, attention and the cached step where byte offsets pass 32 bits (rows
far apart in one large buffer), and calls that name their stream."""
from __future__ import annotations

import sys

import pytest
import torch

import input_dependent_depthwise_amd as dc
from tests import attn_util as au

pytestmark = pytest.mark.gpu


def _note(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def test_rows_past_4_gib():
    """A row of 9000 tokens 512 KiB apart (4.7 GB): forward, backward, rotary, by views of the buffer."""
    _note("[offsets] rows")
    T, H, G, hd = 9000, 4, 2, 64
    buf = torch.empty(1, T, 4096, hd, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    row = torch.randn(1, T, H + 2 * G, hd, generator=g, device="cuda").bfloat16()
    d_o = torch.randn(1, T, H, hd, generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, 3000, 8000, 8990], dtype=torch.int32, device="cuda")
    f = dc.dynconv_rope_freqs(hd)
    far = buf[:, :, 1000:1000 + H + 2 * G]
    far.copy_(row)
    qk = dc.dynconv_rope(row[:, :, :H + G], f, cu_seqlens=cu)
    dc.dynconv_rope(far[:, :, :H + G], f, cu_seqlens=cu, out=far[:, :, :H + G])
    assert torch.equal(far[:, :, :H + G], qk)
    q, k, v = far[:, :, :H], far[:, :, H:H + G], far[:, :, H + G:]
    o, lse = dc.dynconv_attn_fwd(q, k, v, cu_seqlens=cu, want_lse=True, o=buf[:, :, 2000:2000 + H])
    near = [t.contiguous() for t in (q, k, v)]
    o1, lse1 = dc.dynconv_attn_fwd(*near, cu_seqlens=cu, want_lse=True)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    grad = buf[:, :, 3000:3000 + H + 2 * G]
    out = {"dq": grad[:, :, :H], "dk": grad[:, :, H:H + G], "dv": grad[:, :, H + G:]}
    dc.dynconv_attn_bwd(q, k, v, o, lse, d_o, cu_seqlens=cu, out=out)
    want = dc.dynconv_attn_bwd(*near, o1, lse1, d_o, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in want)
    ref = au.attention(*near, cu=cu.tolist())["o"]
    assert au.rel(o1, ref) <= au.TOL["bf16"]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_cache(dtype):
    """A cache whose rows lie 32 or 64 KiB apart: the last ones past 4 GiB, in stretches of their own."""
    _note(f"[offsets] cache {dtype}")
    S, H, G, hd = 140000, 4, 2, 64
    buf = torch.empty(1, S, 256, hd, dtype=au.DTYPES[dtype], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = buf[:, :, 10:10 + G], buf[:, :, 200:200 + G]
    n = 139000
    for c in (kc, vc):
        c.fill_(float("nan"))
        c[:, :n] = torch.randn(1, n, G, hd, generator=g, device="cuda").to(c.dtype)
    new = torch.randn(1, H + 2 * G, hd, generator=g, device="cuda").to(kc.dtype)
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    q, k, v = new[:, :H], new[:, H:H + G], new[:, H + G:]
    o = dc.dynconv_attn_decode(q, k, v, kc, vc, lengths)
    keys = torch.cat((kc[:, :n], k[:, None]), 1).double()
    values = torch.cat((vc[:, :n], v[:, None]), 1).double()
    per = H // G
    for h in range(H):
        p = (keys[0, :, h // per] @ q[0, h].double() * hd ** -0.5).softmax(0)
        assert au.rel(o[0, h], p @ values[0, :, h // per]) <= (2.0 ** -8 if dtype == "bf16" else 1e-5)
    assert torch.equal(kc[0, n], k[0]) and torch.equal(vc[0, n], v[0])
    assert bool(torch.isnan(kc[0, n + 1:]).all())


def test_named_stream():
    """stream=: the work, and what the call allocates, belong to that stream."""
    _note("[offsets] stream")
    g = torch.Generator(device="cuda").manual_seed(3)
    row = torch.randn(2, 400, 8, 64, generator=g, device="cuda").bfloat16()
    d_o = torch.randn(2, 400, 4, 64, generator=g, device="cuda").bfloat16()
    f = dc.dynconv_rope_freqs(64)

    def steps(**kw):
        qk = dc.dynconv_rope(row[:, :, :6], f, **kw)
        q, k, v = qk[:, :, :4], qk[:, :, 4:], row[:, :, 6:]
        o, lse = dc.dynconv_attn_fwd(q, k, v, want_lse=True, **kw)
        grads = dc.dynconv_attn_bwd(q, k, v, o, lse, d_o, **kw)
        kc, vc = k.clone(), v.clone()
        n = torch.tensor([399, 5], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        step = dc.dynconv_attn_decode(q[:, 7], k[:, 7], v[:, 7], kc, vc, n, freqs=f, **kw)
        return [qk, o, lse, *grads.values(), step, kc, vc]

    want = steps()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = []
        for _ in range(2):
            got.append(steps(stream=s))
        torch.cuda.synchronize()
        for out in got:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
