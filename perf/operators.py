"""The operators of the Q/K/V path that follows the short convolution, as cases to measure.

The layer's Q/K/V workloads end where the convolved row ``[B, T, (n_heads + 2 n_kv) head_dim]`` is
written.  What a model does next with that row is measured here:

* ``rope``    rotary positions on the query and key heads of the row (and its inverse, the backward)
* ``prompt``  causal attention over whole prompts, heads in groups, packed documents
* ``train``   the same with its backward: o, dq, dk, dv
* ``decode``  one token for each sequence: rotate q and k, append k and v to the cache, attend

``run`` computes them in elementary torch operations in fp32, rounded once, or, where ``own`` is true,
through the package's entry points.  Definitions (i a query token, j a key token of the same document):

    rope     angle(p, m) = p f[m];  (a, b) -> c (a cos - b sin, b cos + a sin), pairs (2m, 2m+1) or (m, m + rot/2)
    attend   s = scale q_i . k_j for j <= i;  p = exp(s - lse_i);  lse_i = log sum_j exp(s);  o_i = sum_j p v_j
    grad     dv_j = sum_i p do_i;  ds = p (do_i . v_j - do_i . o_i);  dq_i = scale sum_j ds k_j;  dk_j = scale sum_i ds q_i

A token of no document (the padding at the end of a packed row), and a sequence whose cache slot is unused
(length -1), have no keys: their outputs are zero.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # the smallest call: one short row of the tiny fp32 workload (4 heads of 16), latency
        dict(name="rope_tiny", kind="rope", dtype="fp32", B=1, T=256, heads=2, kv_heads=2, head_dim=16, rot=16,
             pairs="half", inverse=False, scaling="none", docs=0, layout=0),
        # the 150M Q/K/V batch: 12 + 12 heads of 64 beside the 12 value heads that stay
        dict(name="rope_150m", kind="rope", dtype="bf16", B=8, T=2048, heads=12, kv_heads=12, head_dim=64, rot=64,
             pairs="interleaved", inverse=False, scaling="linear", docs=0, layout=0),
        # the 2B grouped-query row in training: gradients turned back, half of each head, packed, long-context scaling
        dict(name="rope_2b_bwd", kind="rope", dtype="bf16", B=1, T=16384, heads=16, kv_heads=4, head_dim=128, rot=64,
             pairs="half", inverse=True, scaling="blend", docs=19, layout=1),
        # one short question to a small model: latency
        dict(name="prompt_short", kind="prompt", dtype="bf16", B=1, T=37, heads=12, kv_heads=12, head_dim=64, docs=0, layout=0),
        # evaluation of the 150M batch
        dict(name="prompt_150m", kind="prompt", dtype="bf16", B=8, T=2048, heads=12, kv_heads=12, head_dim=64, docs=0, layout=0),
        # the 2B grouped-query batch
        dict(name="prompt_2b", kind="prompt", dtype="bf16", B=4, T=4096, heads=16, kv_heads=4, head_dim=128, docs=0, layout=0),
        # prompts of many lengths in one row of 16384 tokens, a padded end
        dict(name="prompt_2b_packed", kind="prompt", dtype="bf16", B=1, T=16384, heads=16, kv_heads=4, head_dim=128, docs=11, layout=2),
        # parity training of the tiny fp32 workload
        dict(name="train_tiny", kind="train", dtype="fp32", B=1, T=256, heads=2, kv_heads=1, head_dim=16, docs=0, layout=0),
        # a training step of the 150M batch
        dict(name="train_150m", kind="train", dtype="bf16", B=8, T=2048, heads=12, kv_heads=12, head_dim=64, docs=0, layout=0),
        # a training step of the 2B model on packed documents
        dict(name="train_2b_packed", kind="train", dtype="bf16", B=1, T=8192, heads=16, kv_heads=4, head_dim=128, docs=5, layout=3),
        # chat with one user: latency
        dict(name="decode_one", kind="decode", dtype="bf16", B=1, S=1024, heads=12, kv_heads=12, head_dim=64, rot=64,
             pairs="half", scaling="none", layout=4),
        # a serving batch: 64 slots of all lengths up to 8191 cached tokens, grouped heads
        dict(name="decode_2b_batch", kind="decode", dtype="bf16", B=64, S=8192, heads=16, kv_heads=4, head_dim=128, rot=128,
             pairs="half", scaling="blend", layout=5),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["rope", "prompt", "train", "decode"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    head_dim = rng.choice([16, 64, 64, 80, 96, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 12])
    heads = kv_heads * rng.choice([1, 1, 2, 4, 7]) if kv_heads < 12 else 12
    c = dict(kind=kind, dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=head_dim, layout=rng.randrange(1 << 20))
    if kind in ("rope", "decode"):
        c.update(rot=rng.choice([head_dim, head_dim, head_dim // 2]), pairs=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear", "blend"]))
    if kind == "decode":
        S = _spread(rng, 1, 16384)
        # at most the largest listed cache
        most = 64 * 8192 * 4 * 128 * 2 // (S * kv_heads * head_dim * BYTES[dtype])
        c.update(B=_spread(rng, 1, max(1, min(96, most))), S=S)
        return c
    packed = rng.random() < 0.5
    if kind == "rope":
        T = _spread(rng, 1, 16384)
        most = 16384 * 20 * 128 * 2 // (T * (heads + kv_heads) * head_dim * BYTES[dtype])
        c.update(inverse=rng.random() < 0.5)
    else:
        # at most the work of the largest listed attention of its kind, and of its scores in fp32
        area = 16 * (16384 ** 2 if kind == "prompt" else 8192 ** 2) // (4 if dtype == "fp32" else 1)
        T = _spread(rng, 1, min(16384, int(math.sqrt(area / heads))))
        most = int(area / (heads * T * T))
    B = 1 if packed else _spread(rng, 1, max(1, min(16, most)))
    c.update(B=B, T=T, docs=_spread(rng, 1, max(1, min(64, T))) if packed else 0)
    return c


# --- what a case stands for in numbers ---------------------------------------------------------


def _doc_offsets(c):
    """Offsets of the packed documents (their last one before the row's end: up to 1/32 of the row is padding)."""
    r = random.Random(c["layout"])
    T, n = c["T"], c["docs"]
    end = T - r.randrange(T // 32 + 1)
    w = [r.expovariate(1.0) + 0.01 for _ in range(n)]
    cuts, acc = [0], 0.0
    for x in w:
        acc += x
        cuts.append(min(end, round(end * acc / sum(w))))
    cuts[-1] = end
    return cuts


def _cached(c):
    """Tokens that each sequence has in its cache: of all lengths; in a batch one slot is unused, one is fresh."""
    r = random.Random(c["layout"])
    S = c["S"]
    n = [min(S - 1, int(S * math.exp(-2.5 * r.random() ** 2))) for _ in range(c["B"])]
    if c["B"] >= 4:
        n[1], n[2] = -1, 0
    return n


def _pairs(c):
    """(query, key) pairs of one head and one row."""
    if c["docs"]:
        cuts = _doc_offsets(c)
        return sum((b - a) * (b - a + 1) // 2 for a, b in zip(cuts, cuts[1:]))
    return c["B"] * c["T"] * (c["T"] + 1) // 2


def work(case):
    c = case
    eb, hd, H, G = BYTES[c["dtype"]], c["head_dim"], c["heads"], c["kv_heads"]
    if c["kind"] == "rope":
        n = c["B"] * c["T"] * (H + G) * hd
        return {"bytes": 2 * n * eb, "flops": 3 * n * c["rot"] // hd}
    if c["kind"] == "decode":
        keys = sum(n + 1 for n in _cached(c) if n >= 0)
        act = sum(n >= 0 for n in _cached(c))
        return {"bytes": eb * hd * (2 * G * keys + 2 * G * act + 2 * H * c["B"]), "flops": 4 * keys * H * hd}
    rows, pairs = c["B"] * c["T"], _pairs(c)
    if c["kind"] == "prompt":
        return {"bytes": eb * hd * rows * (2 * H + 2 * G) + 4 * rows * H, "flops": 4 * pairs * H * hd}
    # forward (2 products) and backward (5: the scores again, dp, dv, dq, dk); q, k, v, do in, o, dq, dk, dv out
    return {"bytes": eb * hd * rows * (4 * H + 4 * G), "flops": 14 * pairs * H * hd}


# --- inputs --------------------------------------------------------------------------------------


def _freqs(rot, scaling):
    """Angular frequencies (radians a token, fp64) and the factor on the rotated pairs."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        return f / 4, 1.0
    if scaling == "blend":  # long waves (over 4096 tokens / 1) slowed 8 times, short ones (under 4096 / 32) kept
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        return f * keep + f / 8 * (1 - keep), 0.1 * math.log(8) + 1
    return f, 1.0


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, hd, H, G, B = DTYPES[c["dtype"]], c["head_dim"], c["heads"], c["kv_heads"], c["B"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=dt) * std).to(dt)

    s = {"case": dict(c)}
    if c["kind"] in ("rope", "decode"):
        f, s["factor"] = _freqs(c["rot"], c["scaling"])
        s["freqs"] = f.cuda()
    if c["kind"] == "decode":
        # q, k, v of the new token lie in one row, as the convolution's decode step writes it
        row = normal(B, H + 2 * G, hd)
        s["q"], s["k"], s["v"] = row[:, :H], row[:, H:H + G], row[:, H + G:]
        s["k_cache"], s["v_cache"] = normal(B, c["S"], G, hd), normal(B, c["S"], G, hd)
        s["lengths"] = torch.tensor(_cached(c), dtype=torch.int32).cuda()
        return s
    row = normal(B, c["T"], H + 2 * G, hd)  # the convolution's output: query, key and value heads side by side
    s["qk"], s["q"], s["k"], s["v"] = row[:, :, :H + G], row[:, :, :H], row[:, :, H:H + G], row[:, :, H + G:]
    s["cu"] = torch.tensor(_doc_offsets(c), dtype=torch.int32).cuda() if c["docs"] else None
    if c["kind"] == "train":
        s["do"] = normal(B, c["T"], H, hd, std=0.1)
    return s


# --- one pass ------------------------------------------------------------------------------------


def run(state):
    s, c = state, state["case"]
    if own:
        import input_dependent_depthwise_amd as dc
        if c["kind"] == "rope":
            return dc.dynconv_rope(s["qk"], s["freqs"], cu_seqlens=s["cu"], interleaved=c["pairs"] == "interleaved",
                                   factor=s["factor"], inverse=c["inverse"])
        if c["kind"] == "decode":
            o = dc.dynconv_attn_decode(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["lengths"], freqs=s["freqs"],
                                       interleaved=c["pairs"] == "interleaved", factor=s["factor"])
            return {"o": o, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        o, lse = dc.dynconv_attn_fwd(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], want_lse=True)
        if c["kind"] == "prompt":
            return {"o": o, "lse": lse}
        g = dc.dynconv_attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], cu_seqlens=s["cu"])
        return {"o": o, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}
    if c["kind"] == "rope":
        pos = _positions(c, s["cu"])
        return _rotate(s["qk"].float(), pos, s, -1.0 if c["inverse"] else 1.0).to(s["qk"].dtype)
    if c["kind"] == "decode":
        return _plain_decode(s)
    return _plain_attention(s)


def _doc_of(c, cu):
    """The document of each token, -1 for the padding."""
    t = torch.arange(c["T"], device=cu.device)
    doc = torch.searchsorted(cu.long(), t, right=True) - 1
    return torch.where(doc < c["docs"], doc, -1)


def _positions(c, cu):
    t = torch.arange(c["T"], device="cuda")
    if cu is None:
        return t
    doc = _doc_of(c, cu)  # the padding counts on from the last document's end
    return t - cu.long()[torch.where(doc < 0, c["docs"], doc)]


def _rotate(x, pos, s, sign):
    """x [..., T, heads, head_dim] in fp32, pos [..., T]."""
    c = s["case"]
    rot = c["rot"]
    a = torch.remainder(pos.double()[..., None] * s["freqs"], 2 * math.pi).float()[..., None, :]
    cos, sin = a.cos() * s["factor"], a.sin() * (s["factor"] * sign)
    if c["pairs"] == "interleaved":
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_attention(s):
    c = s["case"]
    B, T, H, G, hd = c["B"], c["T"], c["heads"], c["kv_heads"], c["head_dim"]
    dt, scale, n = s["q"].dtype, c["head_dim"] ** -0.5, c["heads"] // c["kv_heads"]
    q = s["q"].float().transpose(1, 2).reshape(B, G, n * T, hd)  # the queries of a group of heads one after another
    k = s["k"].float().transpose(1, 2).contiguous()
    v = s["v"].float().transpose(1, 2).contiguous()
    t = torch.arange(T, device="cuda")
    seen = t[:, None] >= t[None]
    if c["docs"]:
        doc = _doc_of(c, s["cu"])
        seen = seen & (doc[:, None] == doc[None]) & (doc[:, None] >= 0)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(scale).view(B, G, n, T, T).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).view(B, H, T)
    p = (p / total.clamp(min=1e-30)).view(B, G, n * T, T)
    o = torch.matmul(p, v)
    back = lambda y, heads: y.reshape(B, heads, T, hd).transpose(1, 2).to(dt)  # noqa: E731
    if c["kind"] == "prompt":
        return {"o": back(o, H), "lse": lse}
    do = s["do"].float().transpose(1, 2).reshape(B, G, n * T, hd)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(2, 3), q)
    return {"o": back(o, H), "dq": back(dq, H), "dk": back(dk, G), "dv": back(dv, G)}


def _plain_decode(s):
    c = s["case"]
    B, S, H, G, hd = c["B"], c["S"], c["heads"], c["kv_heads"], c["head_dim"]
    dt, n = s["q"].dtype, s["lengths"].long()
    live = (n >= 0) & (n < S)
    at, rows = n.clamp(0, S - 1), torch.arange(B, device="cuda")
    q = _rotate(s["q"].float(), n, s, 1.0).view(B, G, H // G, hd)
    k = _rotate(s["k"].float(), n, s, 1.0).to(dt)
    for_row = live[:, None, None]
    s["k_cache"][rows, at] = torch.where(for_row, k, s["k_cache"][rows, at])
    s["v_cache"][rows, at] = torch.where(for_row, s["v"], s["v_cache"][rows, at])
    kc, vc = s["k_cache"].float().transpose(1, 2), s["v_cache"].float().transpose(1, 2)
    x = torch.matmul(q, kc.transpose(2, 3)) * hd ** -0.5
    seen = (torch.arange(S, device="cuda") <= n[:, None]) & live[:, None]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    o = torch.matmul(p, vc) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return {"o": o.view(B, H, hd).to(dt), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# --- the definitions in 64 bits ------------------------------------------------------------------


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "rope":
        pos = torch.arange(c["T"], dtype=torch.float64)
        if c["docs"]:
            for first in _doc_offsets(c)[1:]:  # counted from the last offset at or before the token
                pos[first:] = torch.arange(c["T"] - first, dtype=torch.float64)
        return _turn64(s, s["qk"].double(), pos.cuda()[None, :, None], -1 if c["inverse"] else 1)
    return _decode64(c, s) if c["kind"] == "decode" else _attention64(c, s)


def _turn64(s, x, pos, sign):
    """Multiplication of each pair, as a complex number, by factor exp(+- i angle).  pos: of x without its last axis."""
    c, rot = s["case"], s["case"]["rot"]
    part = x[..., :rot]
    part = part.unflatten(-1, (rot // 2, 2)) if c["pairs"] == "interleaved" else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    angle = sign * pos[..., None] * s["freqs"]
    z = torch.view_as_complex(part.contiguous()) * torch.polar(torch.full_like(angle, s["factor"]), angle)
    z = torch.view_as_real(z)
    z = z if c["pairs"] == "interleaved" else z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), x[..., rot:]), -1)


def _attention64(c, s):
    T, H, n, hd = c["T"], c["heads"], c["heads"] // c["kv_heads"], c["head_dim"]
    q, k, v = (s[x].double() for x in "qkv")
    out = {"o": torch.zeros_like(q)}
    lse = torch.full((c["B"], H, T), -math.inf, dtype=torch.float64, device="cuda")
    if c["kind"] == "train":
        do = s["do"].double()
        out.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    cuts = _doc_offsets(c) if c["docs"] else [0, T]
    for b in range(c["B"]):
        for lo, hi in zip(cuts, cuts[1:]):
            above = torch.ones(hi - lo, hi - lo, dtype=torch.bool, device="cuda").triu(1)
            for h in range(H if hi > lo else 0):
                d, g = slice(lo, hi), h // n
                x = (q[b, d, h] @ k[b, d, g].T) / math.sqrt(hd)
                x.masked_fill_(above, -math.inf)
                lse[b, h, d] = x.logsumexp(-1)
                x = x.sub_(lse[b, h, d, None]).exp_()
                out["o"][b, d, h] = x @ v[b, d, g]
                if c["kind"] == "train":
                    out["dv"][b, d, g] += x.T @ do[b, d, h]
                    x *= do[b, d, h] @ v[b, d, g].T - (do[b, d, h] * out["o"][b, d, h]).sum(-1, keepdim=True)
                    out["dq"][b, d, h] = x @ k[b, d, g] / math.sqrt(hd)
                    out["dk"][b, d, g] += x.T @ q[b, d, h] / math.sqrt(hd)
    return {"o": out["o"], "lse": lse} if c["kind"] == "prompt" else out


def _decode64(c, s):
    # the cache holds rounded keys: the appended one is rounded as it is stored before it is attended to
    dt, H, per = DTYPES[c["dtype"]], c["heads"], c["heads"] // c["kv_heads"]
    pos = s["lengths"].double()[:, None]
    q, k = _turn64(s, s["q"].double(), pos, 1), _turn64(s, s["k"].double(), pos, 1)
    o = torch.zeros_like(q)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for b, n in enumerate(_cached(c)):
        if n < 0:
            continue
        kc[b, n], vc[b, n] = k[b], s["v"][b].double()
        for h in range(H):
            keys = kc[b, :n + 1, h // per].clone()
            keys[n] = keys[n].to(dt).double()
            o[b, h] = (keys @ q[b, h] / math.sqrt(c["head_dim"])).softmax(0) @ vc[b, :n + 1, h // per]
    return {"o": o, "k_cache": kc, "v_cache": vc}
