"""Rotary positions (dynconv_rope) against complex multiplication in fp64: both
pairings, parts of a head, widths that take the 16-byte, 8-byte and
single-element kernels, positions given, of documents and far out, in place,
the inverse as the backward."""
from __future__ import annotations

import sys

import pytest
import torch

import input_dependent_depthwise_amd as dc
from tests import attn_util as au

pytestmark = pytest.mark.gpu

# one rounding of the result (2^-8 of each element at most); fp32: the angle, sine and
# cosine to 2^-23 or so each, two products and a sum
TOL = {"bf16": 2.0 ** -8, "fp32": 5e-7}


def _note(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _x(B, T, H, hd, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(B, T, H, hd, generator=g, device="cuda").to(au.DTYPES[dtype])


def _index(B, T):
    return torch.arange(T, device="cuda").expand(B, T)


SHAPES = [
    # B, T, H, hd, rot
    (1, 1, 1, 2, 2),
    (2, 7, 3, 16, 16),
    (1, 100, 4, 16, 8),
    (2, 33, 5, 64, 64),
    (1, 300, 24, 64, 32),
    (3, 129, 20, 128, 128),
    (1, 1025, 20, 128, 64),
    (2, 50, 3, 80, 40),
    (2, 50, 3, 96, 48),
    (1, 61, 7, 10, 6),
    (1, 61, 7, 72, 22),
    (1, 17, 2, 48, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_definition(shape, interleaved, dtype):
    _note(f"[rope] {shape} interleaved={interleaved} {dtype}")
    B, T, H, hd, rot = shape
    x = _x(B, T, H, hd, dtype, seed=sum(shape))
    f = dc.dynconv_rope_freqs(rot)
    for inverse in (False, True):
        y = dc.dynconv_rope(x, f, interleaved=interleaved, factor=1.25, inverse=inverse)
        ref = au.rotate(x, f, _index(B, T), interleaved, 1.25, inverse)
        assert au.rel(y, ref) <= TOL[dtype]
        assert torch.equal(y[..., rot:], x[..., rot:])
        z = x.clone()
        assert dc.dynconv_rope(z, f, interleaved=interleaved, factor=1.25, inverse=inverse, out=z) is z
        assert torch.equal(z, y)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
def test_positions(interleaved, dtype):
    """Given positions, negative and up to 2^31 - 1: the angle is reduced in fp64 (2^31 positions at
    2^-53: below 2^-22 turns), the definition's own angle in fp64 likewise."""
    _note(f"[rope] positions {dtype}")
    x = _x(2, 40, 6, 64, dtype, seed=3)
    f = dc.dynconv_rope_freqs(64)
    pos = torch.randint(-(1 << 20), 1 << 20, (2, 40), dtype=torch.int32, device="cuda")
    pos[0, :3] = torch.tensor([2 ** 31 - 1, -(2 ** 31), 0], dtype=torch.int32)
    y = dc.dynconv_rope(x, f, positions=pos, interleaved=interleaved)
    assert au.rel(y, au.rotate(x, f, pos, interleaved)) <= max(TOL[dtype], 2e-6)


@pytest.mark.parametrize("cu", [[0, 5, 5, 6, 100, 131], [0, 200], [0, 0, 64, 128, 190]], ids=str)
def test_documents(cu):
    T = 200
    _note(f"[rope] documents {cu}")
    x = _x(1, T, 4, 128, "fp32", seed=4)
    f = dc.dynconv_rope_freqs(128, 500000.0)
    pos = torch.zeros(1, T, dtype=torch.int64, device="cuda")
    for lo in cu:
        pos[0, lo:] = torch.arange(T - lo, device="cuda")
    y = dc.dynconv_rope(x, f, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert au.rel(y, au.rotate(x, f, pos)) <= TOL["fp32"]


def test_views_and_backward():
    """The query and key heads of a row, in place, leave the value heads; turning back undoes it
    and is its transpose."""
    _note("[rope] views")
    row = _x(2, 77, 16, 64, "fp32", seed=5)
    keep = row.clone()
    f = dc.dynconv_rope_freqs(64)
    dc.dynconv_rope(row[:, :, :12], f, out=row[:, :, :12])
    assert torch.equal(row[:, :, 12:], keep[:, :, 12:])
    assert au.rel(row[:, :, :12], au.rotate(keep[:, :, :12], f, _index(2, 77))) <= TOL["fp32"]
    back = dc.dynconv_rope(row[:, :, :12], f, inverse=True)
    assert au.rel(back, keep[:, :, :12]) <= 2 * TOL["fp32"]
    g = _x(2, 77, 12, 64, "fp32", seed=6)
    a = (row[:, :, :12].double() * g.double()).sum()
    b = (keep[:, :, :12].double() * dc.dynconv_rope(g, f, inverse=True).double()).sum()
    assert abs((a - b).item()) <= 1e-6 * row[:, :, :12].double().norm().item() * g.double().norm().item()
    hm = keep.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(dc.dynconv_rope(hm, f), dc.dynconv_rope(keep, f))


def test_frequencies():
    f = dc.dynconv_rope_freqs(64, 10000.0, device="cpu")
    want = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    assert torch.allclose(f, want, rtol=1e-14)
    assert torch.allclose(dc.dynconv_rope_freqs(64, stretch=4.0, device="cpu"), want / 4, rtol=1e-14)
    g = dc.dynconv_rope_freqs(64, stretch=8.0, trained_len=4096, slow_turns=1.0, fast_turns=32.0, device="cpu")
    turns = 4096 * want / (2 * torch.pi)
    assert torch.allclose(g[turns >= 32], want[turns >= 32], rtol=1e-14)
    assert torch.allclose(g[turns <= 1], want[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert bool(((g[mid] > want[mid] / 8) & (g[mid] < want[mid])).all())


def test_empty():
    f = dc.dynconv_rope_freqs(64)
    x = torch.empty(1, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert dc.dynconv_rope(x, f).shape == x.shape
