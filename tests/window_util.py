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


def paged_rows(table, n_pages, size, b, positions):
    """(rows of the pool, which of them exist) of the given positions of sequence b."""
    page = table[b].long()[positions // size]
    ok = (page >= 0) & (page < n_pages)
    return torch.where(ok, page, 0) * size + positions % size, ok


def paged_decode(q, k_row, v, kp, vp, table, lengths, window=None, sinks=0, scale=None, freqs=None, interleaved=False,
                 factor=1.0):
    """o of one step over pools as they are before it, in fp64.  k_row [B, G, hd]: the new keys as they are stored."""
    B, H, hd = q.shape
    G, (n_pages, size) = k_row.shape[1], kp.shape[:2]
    scale = 1 / math.sqrt(hd) if scale is None else scale
    q = q.double()
    if freqs is not None:
        q = au.rotate(q[:, None].cpu(), freqs.cpu(), lengths.view(B, 1).cpu(), interleaved, factor)[:, 0].to(q.device)
    o = torch.zeros_like(q)
    for b, n in enumerate(lengths.tolist()):
        if n < 0 or n >= table.shape[1] * size:
            continue
        j = torch.arange(n, device=q.device)
        if window is not None:
            j = j[(n - j < window) | (j < sinks)]
        rows, ok = paged_rows(table, n_pages, size, b, j)
        keys = torch.cat((kp.flatten(0, 1)[rows[ok]], k_row[b:b + 1].to(kp.dtype))).double()
        values = torch.cat((vp.flatten(0, 1)[rows[ok]], v[b:b + 1])).double()
        for h in range(H):
            g = h // (H // G)
            s = keys[:, g] @ q[b, h] * scale
            if bool((s == -math.inf).all()):
                continue
            o[b, h] = au.seen_product(s.softmax(0)[None], values[:, g], (s == -math.inf)[None])[0]
    return o
