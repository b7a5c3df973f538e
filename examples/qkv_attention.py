"""A Q/K/V attention layer from its hidden state to its output, as a model would run it.

    python examples/qkv_attention.py

Projection and dynamic short convolution (``dynconv_fwd_proj``, ``DynConvFn``), rotary positions and
causal attention with grouped heads (``QKVAttnFn``): a few training steps on packed documents, then the
same layer one token at a time (``dynconv_decode``, ``dynconv_attn_decode``) against the whole prompt.
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

    def train(self, h, cu_seqlens=None):
        """h [B, T, d] -> o [B, T, n_heads, head_dim], with gradients."""
        x = h @ self.Wp
        row = dc.DynConvFn.apply(h, x, self.W, None, None, self.w0, self.k, self.groups, cu_seqlens)
        return dc.QKVAttnFn.apply(row, self.H, self.G, self.freqs, False, 1.0, None, cu_seqlens)

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


def train(steps=8):
    """Gradient descent towards another layer's outputs on a packed row; returns the losses."""
    d, heads = 256, dict(n_heads=4, n_kv_heads=2, head_dim=64)
    layer, teacher = Layer(d, **heads, seed=1), Layer(d, **heads, seed=2)
    cu = torch.tensor([0, 70, 71, 200, 384], dtype=torch.int32, device="cuda")
    h = torch.randn(1, 384, d, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    target = teacher.train(h, cu).detach().float()
    losses = []
    for _ in range(steps):
        loss = (layer.train(h, cu).float() - target).square().mean()
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


if __name__ == "__main__":
    losses = train()
    print("training losses:", ", ".join(f"{x:.5f}" for x in losses))
    off, size = decode()
    print(f"prompt and steps against the whole prompt: at most {off:.4f} apart (largest output {size:.3f})")
