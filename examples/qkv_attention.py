"""A Q/K/V attention layer from its hidden state to its output, as a model would run it.

    python examples/qkv_attention.py

Projection and dynamic short convolution (``dynconv_fwd_proj``, ``DynConvFn``), rotary positions and
causal attention with grouped heads (``QKVAttnFn``): a few training steps on packed documents, then the
same layer one token at a time (``dynconv_decode``, ``dynconv_attn_decode``) against the whole prompt.  Then
the same for long contexts: attention through a sliding window with sinks (``QKVAttnFn`` with a window), and
ragged sequences served from a cache kept in pages (``dynconv_attn_paged_store``, ``dynconv_attn_paged_decode``),
whose pages are given back as the window leaves them.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import input_dependent_depthwise_amd as dc  # noqa: E402


class Layer:
    """Weights of one layer: projection Wp, head-wise filter generator W, bias w0."""

    def __init__(self, d, n_heads, n_kv_heads, head_dim, k=4, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.G, self.hd, self.k = n_heads, n_kv_heads, head_dim, k
        self.groups = n_heads + 2 * n_kv_heads  # one filter a head

        def draw(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype).requires_grad_()

        self.Wp = draw(d, self.groups * head_dim, std=d ** -0.5)
        self.W = draw(d, self.groups * k, std=0.3 * d ** -0.5)
        self.w0 = draw(self.groups * head_dim, k, std=0.1)
        self.freqs = dc.dynconv_rope_freqs(head_dim)

    def train(self, h, cu_seqlens=None, window=None, sinks=0):
        """h [B, T, d] -> o [B, T, n_heads, head_dim], with gradients."""
        x = h @ self.Wp
        row = dc.DynConvFn.apply(h, x, self.W, None, None, self.w0, self.k, self.groups, cu_seqlens)
        return dc.QKVAttnFn.apply(row, self.H, self.G, self.freqs, False, 1.0, None, cu_seqlens, window, sinks)

    @torch.no_grad()
    def prompt(self, h):
        """The whole prompt at once: o and the caches (history of x, keys and values) to go on from."""
        H, G = self.H, self.G
        x, row = dc.dynconv_fwd_proj(h, self.Wp, k=self.k, W=self.W, w0=self.w0, n_heads=self.groups)
        heads = row.view(*row.shape[:2], H + 2 * G, self.hd)
        qk, v = dc.dynconv_rope(heads[:, :, :H + G], self.freqs), heads[:, :, H + G:]
        return dc.dynconv_attn_fwd(qk[:, :, :H], qk[:, :, H:], v), x, qk[:, :, H:], v

    @torch.no_grad()
    def step(self, h, state, k_cache, v_cache, lengths):
        """One token per sequence: h [B, d] -> o [B, n_heads, head_dim]; state and caches updated in place."""
        H, G = self.H, self.G
        x = h @ self.Wp
        row = dc.dynconv_decode(h, x, state, k=self.k, W=self.W, w0=self.w0, n_heads=self.groups)
        heads = row.view(-1, H + 2 * G, self.hd)
        return dc.dynconv_attn_decode(heads[:, :H], heads[:, H:H + G], heads[:, H + G:], k_cache, v_cache, lengths,
                                      freqs=self.freqs)

    @torch.no_grad()
    def row(self, h):
        """The convolved heads [B, T, n_heads + 2 n_kv_heads, head_dim] of h, and the convolution's inputs x."""
        x, row = dc.dynconv_fwd_proj(h, self.Wp, k=self.k, W=self.W, w0=self.w0, n_heads=self.groups)
        return row.view(*row.shape[:2], self.groups, self.hd), x

    @torch.no_grad()
    def step_paged(self, h, state, k_pages, v_pages, table, lengths, window, sinks):
        """step() over a cache kept in pages."""
        H, G = self.H, self.G
        x = h @ self.Wp
        heads = dc.dynconv_decode(h, x, state, k=self.k, W=self.W, w0=self.w0, n_heads=self.groups).view(-1, self.groups, self.hd)
        return dc.dynconv_attn_paged_decode(heads[:, :H], heads[:, H:H + G], heads[:, H + G:], k_pages, v_pages, table,
                                            lengths, window=window, sinks=sinks, freqs=self.freqs)


def train(steps=8, window=None, sinks=0):
    """Gradient descent towards another layer's outputs on a packed row; returns the losses."""
    d, heads = 256, dict(n_heads=4, n_kv_heads=2, head_dim=64)
    layer, teacher = Layer(d, **heads, seed=1), Layer(d, **heads, seed=2)
    cu = torch.tensor([0, 70, 71, 200, 384], dtype=torch.int32, device="cuda")
    h = torch.randn(1, 384, d, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    target = teacher.train(h, cu, window, sinks).detach().float()
    losses = []
    for _ in range(steps):
        loss = (layer.train(h, cu, window, sinks).float() - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for w in (layer.Wp, layer.W, layer.w0):
                g = w.grad.float()
                w -= (0.02 * w.float().norm() / g.norm() * g).to(w.dtype)
                w.grad = None
        losses.append(loss.item())
    return losses


def decode(prompt=40, more=24):
    """A prompt at once, then `more` tokens one by one; the largest difference from all of it at once."""
    d, B = 256, 3
    layer = Layer(d, n_heads=8, n_kv_heads=2, head_dim=128, seed=5)
    h = torch.randn(B, prompt + more, d, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").bfloat16()
    whole = layer.prompt(h)[0]
    o, x, keys, values = layer.prompt(h[:, :prompt].contiguous())
    state = x[:, prompt - layer.k + 1:].contiguous()
    caches = [torch.zeros(B, 128, layer.G, layer.hd, dtype=h.dtype, device="cuda") for _ in range(2)]
    for cache, filled in zip(caches, (keys, values)):
        cache[:, :prompt] = filled
    lengths = torch.full((B,), prompt, dtype=torch.int32, device="cuda")
    steps = [o]
    for t in range(prompt, prompt + more):
        steps.append(layer.step(h[:, t].contiguous(), state, *caches, lengths)[:, None])
        lengths += 1
    return (torch.cat(steps, 1).float() - whole.float()).abs().max().item(), whole.float().abs().max().item()


def serve(prompts=(40, 130, 7), more=60, window=48, sinks=2, size=16):
    """Ragged prompts into pages, then tokens one by one, pages handed out when a sequence needs one and given back when its
    window has left them; the largest difference from each whole row through the window, its size, and the most pages in use."""
    d, B = 256, len(prompts)
    layer = Layer(d, n_heads=8, n_kv_heads=2, head_dim=128, seed=7)
    H, G = layer.H, layer.G
    g = torch.Generator(device="cuda").manual_seed(8)
    longest = max(prompts)
    h = torch.randn(B, longest + more, d, generator=g, device="cuda").bfloat16()
    whole, _ = layer.row(h)
    qk = dc.dynconv_rope(whole[:, :, :H + G], layer.freqs)
    whole = dc.dynconv_attn_window_fwd(qk[:, :, :H], qk[:, :, H:], whole[:, :, H + G:], window, sinks=sinks)

    per_seq = -(-(longest + more) // size)
    pools = [torch.zeros(B * per_seq, size, G, layer.hd, dtype=h.dtype, device="cuda") for _ in range(2)]
    free, table = list(range(B * per_seq)), [[-1] * per_seq for _ in range(B)]
    for b, n in enumerate(prompts):
        for j in range(n // size + 1):
            table[b][j] = free.pop()
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    heads, x = layer.row(h[:, :longest].contiguous())
    pages = torch.tensor(table, dtype=torch.int32, device="cuda")
    dc.dynconv_attn_paged_store(heads[:, :, H:H + G], heads[:, :, H + G:], *pools, pages, counts=lengths, freqs=layer.freqs)
    # (a prompt shorter than the taps has zeros before it)
    pad = torch.cat((torch.zeros(B, layer.k - 1, x.shape[2], dtype=x.dtype, device="cuda"), x), 1)
    state = torch.stack([pad[b, n:n + layer.k - 1] for b, n in enumerate(prompts)])
    off, size_of, most = 0.0, 0.0, 0
    for t in range(more):
        new = torch.stack([h[b, n + t] for b, n in enumerate(prompts)])
        o = layer.step_paged(new, state, *pools, pages, lengths, window, sinks)
        for b, n in enumerate(prompts):
            off = max(off, (o[b].float() - whole[b, n + t].float()).abs().max().item())
            size_of = max(size_of, o[b].float().abs().max().item())
            at = n + t + 1  # the next token's position
            if table[b][at // size] < 0:
                table[b][at // size] = free.pop()
            for j in range(-(-sinks // size), max(0, at + 1 - window) // size):
                if table[b][j] >= 0:
                    free.append(table[b][j])
                    table[b][j] = -1
        lengths += 1
        pages.copy_(torch.tensor(table, dtype=torch.int32))
        most = max(most, B * per_seq - len(free))
    return off, size_of, most


if __name__ == "__main__":
    losses = train()
    print("training losses:", ", ".join(f"{x:.5f}" for x in losses))
    off, size = decode()
    print(f"prompt and steps against the whole prompt: at most {off:.4f} apart (largest output {size:.3f})")
    losses = train(window=40, sinks=2)
    print("training losses through a window of 40 tokens and 2 sinks:", ", ".join(f"{x:.5f}" for x in losses))
    off, size, pages = serve()
    print(f"prompts in pages and steps through a window against the whole rows: at most {off:.4f} apart (largest output "
          f"{size:.3f}), {pages} pages in use at most")
