"""Plain fp64 definitions of attention through a window with sinks and of the paged cache, written with loops over
heads and documents, for the GPU tests."""
from __future__ import annotations

import math

import torch

from tests import attn_util as au


def hidden_pairs(n, window, sinks, device="cuda"):
    """[n, n]: whether token i (row) of a document does not see token j."""
    i, j = torch.arange(n, device=device)[:, None], torch.arange(n, device=device)[None]
    return (j > i) | ((i - j >= window) & (j >= sinks))


def attention(q, k, v, window, sinks=0, scale=None, cu=None, d_o=None):
    """As attn_util.attention, through a window."""
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
            d, hidden = slice(lo, hi), hidden_pairs(hi - lo, window, sinks, q.device)
            for h in range(H if hi > lo else 0):
                g = h // n
                s = (q[b, d, h] @ k[b, d, g].T * scale).masked_fill(hidden, -math.inf)
                r["lse"][b, h, d] = s.logsumexp(-1)
                p = (s - s.logsumexp(-1, keepdim=True)).exp().masked_fill(hidden, 0.0)
                r["o"][b, d, h] = au.seen_product(p, v[b, d, g], hidden)
                if d_o is not None:
                    do = d_o[b, d, h]
                    dp = do @ v[b, d, g].T - (do * r["o"][b, d, h]).sum(-1, keepdim=True)
                    ds = (p * dp).masked_fill(hidden, 0.0) * scale
                    r["dv"][b, d, g] += au.seen_product(p.T, do, hidden.T)
                    r["dq"][b, d, h] = au.seen_product(ds, k[b, d, g], hidden)
                    r["dk"][b, d, g] += au.seen_product(ds.T, q[b, d, h], hidden.T)
                    size = do.abs() @ v[b, d, g].abs().T + (do * r["o"][b, d, h]).abs().sum(-1, keepdim=True)
                    size = (p * size).masked_fill(hidden, 0.0) * scale
                    r["~dq"] += (size @ k[b, d, g].abs()).square().sum().item()
                    r["~dk"] += (size.T @ q[b, d, h].abs()).square().sum().item()
    for name in ("~dq", "~dk"):
        if name in r:
            r[name] = math.sqrt(r[name])
    return r
