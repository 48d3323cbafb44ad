"""Plain 64-bit definitions of the rotary positions, of attention with modified scores and masks, and of the eviction
from a cache, written apart from the library: loops over sequences, dense masks, explicit formulas."""
import math

import torch

TWO_PI = 2 * math.pi


def rope(x, positions, freqs, interleaved, magnitude=1.0):
    """x [N, heads, dims] turned in 64 bits; the angle from exact integers (position * freq modulo 2^64)."""
    half = freqs.numel()
    n = x.shape[0]
    angle = torch.empty((n, half), dtype=torch.float64)
    for j, p in enumerate(positions.tolist()):
        for i, f in enumerate(freqs.tolist()):
            turn = (p * f) % (1 << 64)
            angle[j, i] = (turn - (1 << 64) if turn >= 1 << 63 else turn) / 2.0 ** 64 * TWO_PI
    cos, sin = (angle.cos() * magnitude)[:, None], (angle.sin() * magnitude)[:, None]
    y = x.detach().cpu().double().clone()
    a, b = ((y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if interleaved else (y[..., :half], y[..., half:2 * half]))
    a, b = a.clone(), b.clone()
    first, second = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = first, second
    else:
        y[..., :half], y[..., half:2 * half] = first, second
    return y


def rope_bound(x, ref, half, interleaved, magnitude=1.0):
    """How far a turned row may be off: half a step of its type, the angle's 2^-23 rad, and fp32 cosines, sines and
    products, (|a| + |b|) times 2^-21 in all; half of fp16's smallest step (bf16's is far below)."""
    y = x.detach().cpu().double().abs()
    a, b = ((y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if interleaved else (y[..., :half], y[..., half:2 * half]))
    size = torch.zeros_like(y)
    if interleaved:
        size[..., 0:2 * half:2] = size[..., 1:2 * half:2] = a + b
    else:
        size[..., :half] = size[..., half:2 * half] = a + b
    return ref.abs() * (torch.finfo(x.dtype).eps / 2) + size * (abs(magnitude) * 2.0 ** -21) + 2.0 ** -25
