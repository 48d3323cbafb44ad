"""The 4-bit cache's definition in 64 bits, for the tests: a quantiser, the byte
format and attention over the values that the cache stands for. Shares no code
with the library; everything is plain torch on whatever device the inputs are."""
import math

import torch

D, GROUP, BS, TILE = 128, 32, 256, 16


def quantise(x):
    """[..., 128] -> codes [..., 128] (int64), s and z [..., 4] (fp16)."""
    g = x.double().unflatten(-1, (4, GROUP))
    finite = torch.isfinite(g).all(-1)
    g = torch.where(torch.isfinite(g), g, torch.zeros_like(g)).clamp(-65504.0, 65504.0)
    lo, hi = g.amin(-1), g.amax(-1)
    z, s = lo.to(torch.float16), ((hi - lo) / 15).to(torch.float16)
    sd = s.double()[..., None]
    code = torch.where(sd > 0, ((g - z.double()[..., None]) / sd.clamp(min=2.0 ** -24)).round(), torch.zeros_like(g))
    nan = torch.full_like(s, float("nan"))
    code = torch.where(finite[..., None], code.clamp(0, 15), torch.zeros_like(code))
    return code.long().flatten(-2), torch.where(finite, s, nan), torch.where(finite, z, nan)


def values(code, s, z):
    """What codes stand for, in 64 bits."""
    return (code.unflatten(-1, (4, GROUP)).double() * s.double()[..., None] + z.double()[..., None]).flatten(-2)


def dequantised(x):
    return values(*quantise(x))


def code_place(d, token, is_v):
    """(byte in the tile, shift) of dim d's code of a token (0..15 in its tile)."""
    j = d // 32
    if is_v:
        r, p = d % 32 // 4, d % 4
        return token * 64 + (r ^ (token & 4)) * 8 + 2 * j + p // 2, 4 * (p % 2)
    t, p = d % 32 // 8, d % 8
    return token * 64 + 16 * t + 4 * j + p // 2, 4 * (p % 2)


def row_bytes(code, s, z, token, is_v):
    """One row (codes [128], s, z [4]) -> {byte in the tile: value} as two tensors (places, bytes)."""
    places, out = [], []
    acc = {}
    for d in range(D):
        at, shift = code_place(d, token, is_v)
        acc[at] = acc.get(at, 0) | (int(code[d]) << shift)
    for j in range(4):
        pair = torch.stack((s[j], z[j])).cpu().view(torch.uint8).tolist()
        for i in range(4):
            acc[TILE * 64 + token * 16 + 4 * j + i] = pair[i]
    for at in sorted(acc):
        places.append(at)
        out.append(acc[at])
    return torch.tensor(places), torch.tensor(out, dtype=torch.uint8)


def attention(q, k, v, first, scale):
    """q [n, hq, 128] at positions first.. over k, v [T, hkv, 128] in 64 bits -> [n, hq, 128]."""
    g = q.shape[1] // k.shape[1]
    kk, vv = k.double().repeat_interleave(g, 1), v.double().repeat_interleave(g, 1)
    s = torch.einsum("nhd,thd->hnt", q.double(), kk) * scale
    pos = first + torch.arange(q.shape[0], device=q.device)
    s = s.masked_fill(torch.arange(k.shape[0], device=q.device) > pos[:, None], -math.inf)
    return torch.einsum("hnt,thd->nhd", torch.softmax(s, -1), vv)


def decode_tolerance(ref, q, k, v, codes_v, s_v, z_v, scale):
    """A bound on the decode's error, element by element.

    The result is rounded once (half a step of its type). Before that:
      p s is rounded to fp16: 2^-11 of each s c, or 2^-25 of the largest p s where
        it is subnormal, times 15 and once per token;
      logits are sums of 128 products in fp32, off by at most 2^-20 of the sum of
        their magnitudes A (128 additions of 2^-24 and a few more), which moves p
        and the sum of p by that much each;
      the exponential and the remaining fp32 sums: 2^-20 of the values."""
    half = torch.finfo(q.dtype).eps / 2
    g = q.shape[1] // k.shape[1]
    span = (codes_v.unflatten(-1, (4, GROUP)).double() * s_v.double()[..., None]).amax((0, -1))   # [hkv, 4]
    top = (15 * s_v.double()).amax(0)
    size = v.double().unflatten(-1, (4, GROUP)).abs().amax((0, -1)) + z_v.double().abs().amax(0) + span
    a = (torch.einsum("nhd,thd->hnt", q.double().abs(), k.double().abs().repeat_interleave(g, 1)) * scale).amax((1, 2))
    a = a.unflatten(0, (-1, g))[..., None]                                                          # [hkv, g, 1]
    n = k.shape[0]
    t = span[:, None] * 2.0 ** -11 + n * top[:, None] * 2.0 ** -25 + size[:, None] * 2.0 ** -20 * (1 + 2 * a)
    t = t.flatten(0, 1).repeat_interleave(GROUP, -1)                                                # [hq, 128]
    return half * (ref.abs() + t) + t + 2.0 ** -25
