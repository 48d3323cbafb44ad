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


def attention_rows(q, k, v, first, scale, softcap=0.0, slopes=None, window=0, starts=None, prefix=0):
    """q [n, hq, d] at positions first, first + 1, ... over keys k, v [T, hkv, d] (position = index), in 64 bits.
    Returns (out [n, hq, d], p [hq, n, T], bound [n, hq, d], off [hq, n]): `off` is how far a score may be off in 32-bit
    arithmetic on exact 16-bit rows, `bound` what that makes in `out` before it is rounded to its type. A sum of d products in 32 bits is off by d * 2^-24 of the sum of their
    sizes at most; cap, bias, exponential and sums add some 2^-21 of a score's size."""
    n, hq, d = q.shape
    T, hkv, _ = k.shape
    dev = q.device
    q, k, v = q.double(), k.double(), v.double()
    k, v = (x.repeat_interleave(hq // hkv, 1) for x in (k, v))
    p_at = first + torch.arange(n, device=dev)
    t_at = torch.arange(T, device=dev)
    seen = (t_at[None] <= p_at[:, None]) | (t_at[None] < prefix)
    if starts is not None:
        seen = seen & (t_at[None] >= starts.to(dev).long()[:, None])
    if window > 0:
        seen = seen & (p_at[:, None] - t_at[None] < window)
    # what is not seen by any row may hold anything
    used = seen.any(0)
    k, v = (torch.where(used[:, None, None], x, torch.zeros_like(x)) for x in (k, v))
    s = torch.einsum("nhd,thd->hnt", q, k) * scale
    size = torch.einsum("nhd,thd->hnt", q.abs(), k.abs()).masked_fill(~seen, 0) * scale
    if softcap > 0:
        s = softcap * torch.tanh(s / softcap)
    if slopes is not None:
        s = s - slopes.double().to(dev)[:, None, None] * (p_at[:, None] - t_at[None]).abs().double()
    s = s.masked_fill(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True) if T else torch.zeros((hq, n, 1), device=dev)
    e = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    out = torch.einsum("hnt,thd->nhd", p, v)
    off = size.amax(-1) * (d * 2.0 ** -24) + 2.0 ** -18                       # [hq, n]: of a score
    return out, p, 2 * off.T[..., None] * torch.einsum("hnt,thd->nhd", p, v.abs()), off


def cache_rows(cache, table, length):
    """The first `length` rows [length, hkv, d] that a block table names."""
    blocks = torch.as_tensor(table[:-(-length // 256)], dtype=torch.long, device=cache.device)
    return cache[blocks].flatten(0, 1)[:length]


def evict_choice(weights, first, recent, budget):
    """The positions of `weights` [n] that stay: plain Python, the largest by (weight, lower position first)."""
    n = len(weights)
    if n <= budget:
        return list(range(n))
    middle = range(first, n - recent)

    def size(t):
        return (1, 0.0) if math.isnan(weights[t]) else (0, weights[t])
    best = sorted(middle, key=size, reverse=True)[:budget - first - recent]   # a stable sort
    return sorted(list(range(first)) + best + list(range(n - recent, n)))
