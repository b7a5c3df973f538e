"""Long contexts at bounded cost: attention through a sliding window, and a cache kept in pages.

A model that is trained on long rows and then serves them pays for every earlier token twice: in the attention
over the row and in the cache that each new token reads.  The operators here bound both:

* ``window``        causal attention over whole rows in which a token sees the last ``window`` tokens and the first
                    ``sinks`` tokens of its document, heads in groups, packed documents
* ``window_train``  the same with its backward: o, dq, dk, dv
* ``store``         the keys (turned by the rotary plan) and values of whole prompts into the pages of a cache
* ``step``          one token for each sequence: rotate q and k, store k and v in its page, attend over the pages
                    listed for the sequence, all of it or through the window

``run`` computes them in elementary torch operations in fp32, rounded once, or, where ``own`` is true, through the
package's entry points.  Definitions (i a query token, j a key token, positions counted in their document):

    sees     j <= i  and  (i - j < window  or  j < sinks)
    attend   s = scale q_i . k_j;  p = exp(s - lse_i);  lse_i = log sum_j exp(s);  o_i = sum_j p v_j  over the j that i sees
    grad     dv_j = sum_i p do_i;  ds = p (do_i . v_j - do_i . o_i);  dq_i = scale sum_j ds k_j;  dk_j = scale sum_i ds q_i
    page     position j of sequence b lies in row j % page_size of page table[b, j // page_size]
    turned   angle(j, m) = j f[m];  (a, b) -> c (a cos - b sin, b cos + a sin), pairs (2m, 2m+1) or (m, m + rot/2)

A token of no document (the padding at the end of a packed row), and a slot without a sequence (length -1), see no
keys: their outputs are zero.  Pages that a window has left behind are given back: their table entries are -1.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one short question to a small model whose window is shorter still: latency
        dict(name="window_short", kind="window", dtype="bf16", B=1, T=37, heads=12, kv_heads=12, head_dim=64, window=16,
             sinks=2, docs=0, layout=0),
        # evaluation of the 150M batch with a window of an eighth of the row
        dict(name="window_150m", kind="window", dtype="bf16", B=8, T=2048, heads=12, kv_heads=12, head_dim=64, window=256,
             sinks=4, docs=0, layout=0),
        # long prompts of the 2B grouped-query model in one row of 16384 tokens, a padded end
        dict(name="window_2b_packed", kind="window", dtype="bf16", B=1, T=16384, heads=16, kv_heads=4, head_dim=128,
             window=1024, sinks=4, docs=3, layout=2),
        # parity training of the tiny fp32 workload
        dict(name="window_train_tiny", kind="window_train", dtype="fp32", B=1, T=256, heads=2, kv_heads=1, head_dim=16,
             window=100, sinks=3, docs=0, layout=0),
        # a training step of the 150M batch
        dict(name="window_train_150m", kind="window_train", dtype="bf16", B=8, T=2048, heads=12, kv_heads=12, head_dim=64,
             window=256, sinks=4, docs=0, layout=0),
        # a training step of the 2B model on packed documents
        dict(name="window_train_2b_packed", kind="window_train", dtype="bf16", B=1, T=8192, heads=16, kv_heads=4,
             head_dim=128, window=1024, sinks=4, docs=2, layout=3),
        # a short prompt into an empty cache: latency
        dict(name="store_short", kind="store", dtype="bf16", B=1, T=37, kv_heads=12, head_dim=64, rot=64, pairs="half",
             scaling="none", page=16, past=0, docs=0, layout=4),
        # the next parts of eleven prompts of the 2B model, behind what their pages hold already
        dict(name="store_2b_packed", kind="store", dtype="bf16", B=1, T=16384, kv_heads=4, head_dim=128, rot=128,
             pairs="half", scaling="blend", page=16, past=8192, docs=11, layout=5),
        # chat with one user: latency
        dict(name="step_one", kind="step", dtype="bf16", B=1, S=1024, heads=12, kv_heads=12, head_dim=64, rot=64,
             pairs="half", scaling="none", page=16, window=0, sinks=0, layout=6),
        # a serving batch: 64 slots of all lengths up to 8191 cached tokens, grouped heads
        dict(name="step_2b_batch", kind="step", dtype="bf16", B=64, S=8192, heads=16, kv_heads=4, head_dim=128, rot=128,
             pairs="half", scaling="blend", page=16, window=0, sinks=0, layout=7),
        # the same slots on long conversations, of which a window and the first tokens are kept
        dict(name="step_2b_window", kind="step", dtype="bf16", B=64, S=32768, heads=16, kv_heads=4, head_dim=128, rot=128,
             pairs="half", scaling="blend", page=64, window=1024, sinks=4, layout=8),
        # one long document of 131071 tokens, questioned by one user
        dict(name="step_2b_long", kind="step", dtype="bf16", B=1, S=131072, heads=16, kv_heads=4, head_dim=128, rot=64,
             pairs="interleaved", scaling="linear", page=32, window=0, sinks=0, layout=9),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["window", "window_train", "store", "step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    head_dim = rng.choice([16, 64, 64, 80, 96, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 12])
    heads = kv_heads * rng.choice([1, 1, 2, 4, 7]) if kv_heads < 12 else 12
    c = dict(kind=kind, dtype=dtype, kv_heads=kv_heads, head_dim=head_dim, layout=rng.randrange(1 << 20))
    if kind != "store":
        c.update(heads=heads)
    if kind in ("store", "step"):
        c.update(rot=rng.choice([head_dim, head_dim, head_dim // 2]), pairs=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear", "blend"]), page=rng.choice([1, 6, 8, 16, 16, 16, 20, 32, 64, 64, 128]))
    row = kv_heads * head_dim * BYTES[dtype]
    if kind == "step":
        S = _spread(rng, 1, 131072)
        # at most the largest listed cache
        c.update(B=_spread(rng, 1, max(1, min(96, 64 * 8192 * 4 * 128 * 2 // (S * row)))), S=S, window=0, sinks=0)
        if rng.random() < 0.5:
            c.update(window=_spread(rng, 1, S), sinks=rng.choice([0, 1, 4, 4, 16, 128]))
        return c
    packed = rng.random() < 0.5
    if kind == "store":
        T = _spread(rng, 1, 16384)
        most = 16384 * 4 * 128 * 2 // (T * row)
        c.update(past=rng.choice([0, _spread(rng, 1, 8192)]))
    else:
        # at most the scores of the largest listed attention of its kind, in fp32 a quarter of them
        area = 16 * (16384 ** 2 if kind == "window" else 8192 ** 2) // (4 if dtype == "fp32" else 1)
        T = _spread(rng, 1, min(16384, int(math.sqrt(area / heads))))
        most = int(area / (heads * T * T))
        c.update(window=_spread(rng, 1, T), sinks=rng.choice([0, 1, 4, 4, 16, 128]))
    c.update(B=1 if packed else _spread(rng, 1, max(1, min(16, most))), T=T,
             docs=_spread(rng, 1, max(1, min(64, T))) if packed else 0)
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
    """Tokens that each sequence of a step has in its cache: of all lengths; in a batch one slot is unused, one is fresh."""
    r = random.Random(c["layout"])
    S = c["S"]
    if c["B"] == 1:
        return [S - 1]
    n = [min(S - 1, int(S * math.exp(-2.5 * r.random() ** 2))) for _ in range(c["B"])]
    if c["B"] >= 4:
        n[1], n[2] = -1, 0
    return n


def _past(c):
    """Tokens that the pages of each sequence of a store hold already."""
    r = random.Random(c["layout"] + 1)
    return [r.randrange(c["past"] + 1) for _ in range(c["docs"] or c["B"])]


def _counts(c):
    """New tokens of each sequence of a store."""
    if c["docs"]:
        cuts = _doc_offsets(c)
        return [b - a for a, b in zip(cuts, cuts[1:])]
    return [c["T"]] * c["B"]


def _used_pages(c):
    """For each sequence, which of its pages a cache has to hold: [sequences, pages of a sequence], truth values."""
    ps = c["page"]
    if c["kind"] == "store":
        ends = np.array([p + n for p, n in zip(_past(c), _counts(c))])
        first = np.arange(max(1, -(-int(ends.max()) // ps))) * ps
        return first[None] < ends[:, None]
    n = np.array(_cached(c))
    first = np.arange(-(-c["S"] // ps)) * ps
    used = first[None] <= n[:, None]  # (the new token's page among them)
    if c["window"]:
        used &= (first[None] < c["sinks"]) | (first[None] + ps > n[:, None] + 1 - c["window"])
    return used


def _table(c, rng):
    """The page table, in random order, and the number of pages (some of them are nobody's)."""
    used = _used_pages(c)
    n = int(used.sum()) + 3
    table = np.full(used.shape, -1, dtype=np.int32)
    table[used] = rng.permutation(n)[:n - 3]
    return table, n


def _pairs(c):
    """(query, key) pairs of one head over the batch."""
    total = 0
    for n in _counts(c):
        i = np.arange(n)
        total += int(np.minimum(i + 1, c["window"] + c["sinks"]).sum())
    return total


def work(case):
    c = case
    eb, hd, G = BYTES[c["dtype"]], c["head_dim"], c["kv_heads"]
    if c["kind"] == "store":
        n = sum(_counts(c)) * G * hd
        return {"bytes": 4 * n * eb, "flops": 3 * n * c["rot"] // hd}
    H = c["heads"]
    if c["kind"] == "step":
        n = [x + 1 for x in _cached(c) if x >= 0]
        keys = sum(min(x, c["window"] + c["sinks"]) if c["window"] else x for x in n)
        return {"bytes": eb * hd * (2 * G * keys + 2 * G * len(n) + 2 * H * c["B"]), "flops": 4 * keys * H * hd}
    rows, pairs = c["B"] * c["T"], _pairs(c)
    if c["kind"] == "window":
        return {"bytes": eb * hd * rows * (2 * H + 2 * G) + 4 * rows * H, "flops": 4 * pairs * H * hd}
    # forward (2 products) and backward (5: the scores again, dp, dv, dq, dk); q, k, v, do in, o, dq, dk, dv out
    return {"bytes": eb * hd * rows * (4 * H + 4 * G), "flops": 14 * pairs * H * hd}


# --- inputs --------------------------------------------------------------------------------------


def _freqs(rot, scaling):
    """Angular frequencies (radians a token, fp64) and the factor on the turned pairs."""
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
    dt, hd, G, B = DTYPES[c["dtype"]], c["head_dim"], c["kv_heads"], c["B"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=dt) * std).to(dt)

    s = {"case": dict(c)}
    if c["kind"] in ("store", "step"):
        f, s["factor"] = _freqs(c["rot"], c["scaling"])
        s["freqs"] = f.cuda()
        table, n = _table(c, np.random.default_rng(seed))
        s["table"] = torch.from_numpy(table).cuda()
        # what the pages hold: earlier tokens, and in rows that are nobody's whatever was there
        s["k_pages"], s["v_pages"] = normal(n, c["page"], G, hd), normal(n, c["page"], G, hd)
    if c["kind"] == "step":
        # q, k, v of the new token lie in one row, as the convolution's decode step writes it
        H = c["heads"]
        row = normal(B, H + 2 * G, hd)
        s["q"], s["k"], s["v"] = row[:, :H], row[:, H:H + G], row[:, H + G:]
        s["lengths"] = torch.tensor(_cached(c), dtype=torch.int32).cuda()
        return s
    s["cu"] = torch.tensor(_doc_offsets(c), dtype=torch.int32).cuda() if c["docs"] else None
    if c["kind"] == "store":
        # the key and value heads of the convolution's output
        row = normal(B, c["T"], 2 * G, hd)
        s["k"], s["v"] = row[:, :, :G], row[:, :, G:]
        s["starts"] = torch.tensor(_past(c), dtype=torch.int32).cuda()
        return s
    H = c["heads"]
    row = normal(B, c["T"], H + 2 * G, hd)  # the convolution's output: query, key and value heads side by side
    s["q"], s["k"], s["v"] = row[:, :, :H], row[:, :, H:H + G], row[:, :, H + G:]
    if c["kind"] == "window_train":
        s["do"] = normal(B, c["T"], H, hd, std=0.1)
    return s


# --- one pass ------------------------------------------------------------------------------------


def run(state):
    s, c = state, state["case"]
    if own:
        import input_dependent_depthwise_amd as dc
        if c["kind"] == "store":
            dc.dynconv_attn_paged_store(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], starts=s["starts"],
                                        cu_seqlens=s["cu"], freqs=s["freqs"], interleaved=c["pairs"] == "interleaved",
                                        factor=s["factor"])
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if c["kind"] == "step":
            o = dc.dynconv_attn_paged_decode(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lengths"],
                                             window=c["window"] or None, sinks=c["sinks"], freqs=s["freqs"],
                                             interleaved=c["pairs"] == "interleaved", factor=s["factor"])
            return {"o": o, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        o, lse = dc.dynconv_attn_window_fwd(s["q"], s["k"], s["v"], c["window"], sinks=c["sinks"], cu_seqlens=s["cu"],
                                            want_lse=True)
        if c["kind"] == "window":
            return {"o": o, "lse": lse}
        g = dc.dynconv_attn_window_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], c["window"], sinks=c["sinks"],
                                       cu_seqlens=s["cu"])
        return {"o": o, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}
    if c["kind"] == "store":
        return _plain_store(s)
    return _plain_step(s) if c["kind"] == "step" else _plain_window(s)


def _rotate(x, pos, s):
    """x [..., heads, head_dim] in fp32, pos [...]."""
    c = s["case"]
    rot = c["rot"]
    a = torch.remainder(pos.double()[..., None] * s["freqs"], 2 * math.pi).float()[..., None, :]
    cos, sin = a.cos() * s["factor"], a.sin() * s["factor"]
    if c["pairs"] == "interleaved":
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_window(s):
    c = s["case"]
    B, T, H, G, hd = c["B"], c["T"], c["heads"], c["kv_heads"], c["head_dim"]
    dt, scale, n = s["q"].dtype, c["head_dim"] ** -0.5, c["heads"] // c["kv_heads"]
    q = s["q"].float().transpose(1, 2).reshape(B, G, n * T, hd)  # the queries of a group of heads one after another
    k = s["k"].float().transpose(1, 2).contiguous()
    v = s["v"].float().transpose(1, 2).contiguous()
    t = torch.arange(T, device="cuda")
    start = torch.zeros_like(t)
    seen = t[:, None] >= t[None]
    if c["docs"]:
        cu = s["cu"].long()
        doc = torch.searchsorted(cu, t, right=True) - 1
        start = cu[doc]
        seen = seen & (doc[:, None] == doc[None]) & (doc[:, None] < c["docs"])
    seen = seen & ((t[:, None] - t[None] < c["window"]) | (t - start < c["sinks"])[None])
    x = torch.matmul(q, k.transpose(2, 3)).mul_(scale).view(B, G, n, T, T).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).view(B, H, T)
    p = (p / total.clamp(min=1e-30)).view(B, G, n * T, T)
    o = torch.matmul(p, v)
    back = lambda y, heads: y.reshape(B, heads, T, hd).transpose(1, 2).to(dt)  # noqa: E731
    if c["kind"] == "window":
        return {"o": back(o, H), "lse": lse}
    do = s["do"].float().transpose(1, 2).reshape(B, G, n * T, hd)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(2, 3), q)
    return {"o": back(o, H), "dq": back(dq, H), "dk": back(dk, G), "dv": back(dv, G)}


def _plain_store(s):
    c = s["case"]
    k, v, t = s["k"], s["v"], torch.arange(c["T"], device="cuda")
    if c["docs"]:
        cu = s["cu"].long()
        t = torch.where(t < cu[-1], t, 0)  # (the padding's tokens do again what the first one does)
        k, v = k[:, t], v[:, t]
        seq = torch.searchsorted(cu, t, right=True)[None] - 1
        pos = s["starts"].long()[seq] + t - cu[seq]
    else:
        seq = torch.arange(c["B"], device="cuda")[:, None].expand(-1, c["T"])
        pos = s["starts"].long()[:, None] + t
    k = _rotate(k.float(), pos, s).to(k.dtype)
    ps, width = c["page"], c["kv_heads"] * c["head_dim"]
    at = (s["table"].long()[seq, pos // ps] * ps + pos % ps).flatten()
    s["k_pages"].view(-1, width)[at] = k.reshape(-1, width)
    s["v_pages"].view(-1, width)[at] = v.reshape(-1, width)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_step(s):
    c = s["case"]
    B, S, H, G, hd, ps = c["B"], c["S"], c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    dt, n = s["q"].dtype, s["lengths"].long()
    live = (n >= 0) & (n < S)
    slots, width = torch.arange(B, device="cuda"), G * hd
    q = _rotate(s["q"].float(), n, s).view(B, G, H // G, hd)
    k = _rotate(s["k"].float(), n, s).to(dt)
    table = s["table"].long()
    kp, vp = s["k_pages"].view(-1, width), s["v_pages"].view(-1, width)
    who = torch.where(live, slots, live.long().argmax())  # (a slot without a sequence does again what another does)
    at = n[who]
    rows = table[who, at // ps] * ps + at % ps
    kp[rows], vp[rows] = k.reshape(B, width)[who], s["v"].reshape(B, width)[who]
    # the positions that are looked at: all, or the first and the last ones
    if c["window"]:
        first_of = (n[:, None] + 1 - c["window"]).clamp(min=min(c["sinks"], S))
        last = first_of + torch.arange(min(c["window"], S), device="cuda")
        j = torch.cat((torch.arange(min(c["sinks"], S), device="cuda").expand(B, -1), last), 1)
    else:
        j = torch.arange(S, device="cuda").expand(B, -1)
    seen = (j <= n[:, None]) & live[:, None]
    page = table.gather(1, (j // ps).clamp(max=table.shape[1] - 1))
    rows = torch.where(seen, page * ps + j % ps, 0)
    kc = kp[rows].view(B, -1, G, hd).float().transpose(1, 2).contiguous()
    vc = vp[rows].view(B, -1, G, hd).float().transpose(1, 2).contiguous()
    x = torch.matmul(q, kc.transpose(2, 3)) * hd ** -0.5
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    o = torch.matmul(p, vc) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return {"o": o.view(B, H, hd).to(dt), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# --- the definitions in 64 bits, one sequence and head at a time ------------------------------------


def exact(case, seed):
    c, s = case, prepare(case, seed)
    with torch.no_grad():
        if c["kind"] == "store":
            return _store64(c, s)
        return _step64(c, s) if c["kind"] == "step" else _window64(c, s)


def _turn64(s, x, pos):
    """x [n, heads, head_dim] at the positions pos [n], as complex numbers."""
    c = s["case"]
    rot, m = c["rot"], torch.arange(c["rot"] // 2, device="cuda")
    one, two = (2 * m, 2 * m + 1) if c["pairs"] == "interleaved" else (m, m + rot // 2)
    turn = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device="cuda"),
                       torch.outer(pos.double(), s["freqs"]))[:, None]
    z = torch.complex(x[..., one], x[..., two]) * turn
    y = x.clone()
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _window64(c, s):
    T, H, n, hd, W = c["T"], c["heads"], c["heads"] // c["kv_heads"], c["head_dim"], c["window"]
    q, k, v = (s[x].double() for x in "qkv")
    out = {"o": torch.zeros_like(q)}
    lse = torch.full((c["B"], H, T), -math.inf, dtype=torch.float64, device="cuda")
    if c["kind"] == "window_train":
        do = s["do"].double()
        out.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    cuts = _doc_offsets(c) if c["docs"] else [0, T]
    for lo, hi in zip(cuts, cuts[1:]):
        m, d = hi - lo, slice(lo, hi)
        # hidden: later tokens, and those before the window unless they are among the first
        hidden = torch.ones(m, m, dtype=torch.bool, device="cuda")
        before = hidden.tril(-W)
        before[:, :c["sinks"]] = False
        hidden = hidden.triu(1) | before
        for b in range(c["B"]):
            for h in range(H if m else 0):
                g = h // n
                x = (q[b, d, h] @ k[b, d, g].T) / math.sqrt(hd)
                x.masked_fill_(hidden, -math.inf)
                lse[b, h, d] = x.logsumexp(-1)
                x = x.sub_(lse[b, h, d, None]).exp_()
                out["o"][b, d, h] = x @ v[b, d, g]
                if c["kind"] == "window_train":
                    out["dv"][b, d, g] += x.T @ do[b, d, h]
                    x *= do[b, d, h] @ v[b, d, g].T - (do[b, d, h] * out["o"][b, d, h]).sum(-1, keepdim=True)
                    out["dq"][b, d, h] = x @ k[b, d, g] / math.sqrt(hd)
                    out["dk"][b, d, g] += x.T @ q[b, d, h] / math.sqrt(hd)
    return {"o": out["o"], "lse": lse} if c["kind"] == "window" else out


def _store64(c, s):
    ps, cuts, table = c["page"], _doc_offsets(c) if c["docs"] else None, s["table"].long()
    kp, vp = s["k_pages"].double().flatten(0, 1), s["v_pages"].double().flatten(0, 1)
    for i, (past, n) in enumerate(zip(_past(c), _counts(c))):
        b, d = (0, slice(cuts[i], cuts[i + 1])) if cuts else (i, slice(0, n))
        pos = past + torch.arange(n, device="cuda")
        rows = table[i, pos // ps] * ps + pos % ps
        kp[rows] = _turn64(s, s["k"][b, d].double(), pos)
        vp[rows] = s["v"][b, d].double()
    return {"k_pages": kp.view(s["k_pages"].shape), "v_pages": vp.view(s["v_pages"].shape)}


def _step64(c, s):
    # the cache holds rounded keys: the new one is rounded as it is stored before it is attended to
    dt, H, per, ps = DTYPES[c["dtype"]], c["heads"], c["heads"] // c["kv_heads"], c["page"]
    q, k = (_turn64(s, s[x].double(), s["lengths"]) for x in "qk")
    o = torch.zeros_like(q)
    kp, vp = s["k_pages"].double().flatten(0, 1), s["v_pages"].double().flatten(0, 1)
    table = s["table"].long()
    for b, n in enumerate(_cached(c)):
        if n < 0:
            continue
        j = torch.arange(n + 1, device="cuda")
        if c["window"]:
            j = j[(n - j < c["window"]) | (j < c["sinks"])]
        rows = table[b, j // ps] * ps + j % ps
        kp[rows[-1]], vp[rows[-1]] = k[b], s["v"][b].double()
        keys, values = kp[rows], vp[rows]
        keys[-1] = keys[-1].to(dt).double()
        for h in range(H):
            o[b, h] = (keys[:, h // per] @ q[b, h] / math.sqrt(c["head_dim"])).softmax(0) @ values[:, h // per]
    return {"o": o, "k_pages": kp.view(s["k_pages"].shape), "v_pages": vp.view(s["v_pages"].shape)}
