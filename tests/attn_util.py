"""Plain fp64 definitions of the Q/K/V path behind the convolution (rotary
positions, causal attention and its gradients, the cached step), written with
loops over heads and documents, for the GPU tests."""
from __future__ import annotations

import math

import torch

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# 2-norm of the error over the 2-norm of the result.  bf16: at most three
# roundings of relative size 2^-8 lie on the way to an output (p or ds, the
# saved o in delta, the output itself).  fp32: sums of some thousand terms at
# 2^-24, amplified a few times by the difference do.v - delta; the bar of the
# rest of the library.
TOL = {"bf16": 3 * 2.0 ** -8, "fp32": 1e-5}


def rel(got, ref, noise: float = 0.0) -> float:
    """2-norm of the difference, less `noise`, over the 2-norm of ref (or the difference where ref is zero)."""
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert bool((torch.isnan(got) == torch.isnan(ref)).all()), "NaN in other places"
    fine = torch.isfinite(ref)
    assert bool((got[~fine & ~torch.isnan(ref)] == ref[~fine & ~torch.isnan(ref)]).all()), "infinities differ"
    assert bool(torch.isfinite(got[fine]).all())
    d, n = max(0.0, (got[fine] - ref[fine]).norm().item() - noise), ref[fine].norm().item()
    return d if n == 0.0 else d / n


def rotate(x, freqs, pos, interleaved=False, factor=1.0, inverse=False):
    """x [B, T, heads, head_dim], pos [B, T]."""
    x = x.double().clone()
    ang = pos.double()[:, :, None, None] * freqs.double() * (-1.0 if inverse else 1.0)
    cos, sin, rot = ang.cos() * factor, ang.sin() * factor, 2 * freqs.numel()
    i0 = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    i1 = i0 + 1 if interleaved else i0 + rot // 2
    a, b = x[..., i0].clone(), x[..., i1].clone()
    x[..., i0], x[..., i1] = a * cos - b * sin, b * cos + a * sin
    return x


def attention(q, k, v, scale=None, cu=None, d_o=None):
    """o, lse (and dq, dk, dv with d_o) in fp64; cu: a list of document offsets.
    Also the 2-norms "~dq" and "~dk" of dq and dk with every product and
    difference in them taken by its size: what fp32 rounding is relative to where
    do.v - delta cancels (a token alone in its document has dq = dk = 0)."""
    q, k, v = q.double(), k.double(), v.double()
    B, T, H, hd = q.shape
    n = H // k.shape[2]
    scale = 1 / math.sqrt(hd) if scale is None else scale
    r = {"o": torch.zeros_like(q), "lse": torch.full((B, H, T), -math.inf, dtype=torch.float64, device=q.device)}
    if d_o is not None:
        d_o = d_o.double()
        r.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
        r.update({"~dq": 0.0, "~dk": 0.0})
    cuts = [0, T] if cu is None else list(cu)
    for b in range(B):
        for lo, hi in zip(cuts, cuts[1:]):
            d = slice(lo, hi)
            later = torch.ones(hi - lo, hi - lo, dtype=torch.bool, device=q.device).triu(1)
            for h in range(H if hi > lo else 0):
                g = h // n
                s = (q[b, d, h] @ k[b, d, g].T * scale).masked_fill(later, -math.inf)
                r["lse"][b, h, d] = s.logsumexp(-1)
                p = (s - s.logsumexp(-1, keepdim=True)).exp().masked_fill(later, 0.0)
                r["o"][b, d, h] = seen_product(p, v[b, d, g], later)
                if d_o is not None:
                    do = d_o[b, d, h]
                    dp = do @ v[b, d, g].T - (do * r["o"][b, d, h]).sum(-1, keepdim=True)
                    ds = (p * dp).masked_fill(later, 0.0) * scale
                    r["dv"][b, d, g] += seen_product(p.T, do, later.T)
                    r["dq"][b, d, h] = seen_product(ds, k[b, d, g], later)
                    r["dk"][b, d, g] += seen_product(ds.T, q[b, d, h], later.T)
                    size = do.abs() @ v[b, d, g].abs().T + (do * r["o"][b, d, h]).abs().sum(-1, keepdim=True)
                    size = (p * size).masked_fill(later, 0.0) * scale
                    r["~dq"] += (size @ k[b, d, g].abs()).square().sum().item()
                    r["~dk"] += (size.T @ q[b, d, h].abs()).square().sum().item()
    for name in ("~dq", "~dk"):
        if name in r:
            r[name] = math.sqrt(r[name])
    return r


def seen_product(p, x, hidden):
    """p @ x where a hidden pair contributes nothing, whatever x holds there."""
    if bool(torch.isfinite(x).all()):
        return p @ x
    out = torch.zeros(p.shape[0], x.shape[1], dtype=p.dtype, device=p.device)
    for i in range(p.shape[0]):
        out[i] = p[i][~hidden[i]] @ x[~hidden[i]]
    return out


def decode(q, k, v, kc, vc, lengths, scale=None, freqs=None, interleaved=False, factor=1.0):
    """One step: (o, k_cache, v_cache) in fp64 (the stored key rounded to the cache's type before it is read)."""
    dt, (B, H, hd), G = kc.dtype, q.shape, k.shape[1]
    scale = 1 / math.sqrt(hd) if scale is None else scale
    pos = lengths.view(B, 1)
    q, k = q.double(), k.double()
    if freqs is not None:
        q = rotate(q[:, None], freqs, pos, interleaved, factor)[:, 0]
        k = rotate(k[:, None], freqs, pos, interleaved, factor)[:, 0]
    kc, vc = kc.double(), vc.double()
    o = torch.zeros_like(q)
    for b, n in enumerate(lengths.tolist()):
        if n < 0 or n >= kc.shape[1]:
            continue
        kc[b, n], vc[b, n] = k[b].to(dt).double(), v[b].double()
        for h in range(H):
            g = h // (H // G)
            o[b, h] = (kc[b, :n + 1, g] @ q[b, h] * scale).softmax(0) @ vc[b, :n + 1, g]
    return o, kc, vc
