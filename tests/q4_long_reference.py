"""Long contexts over the 4-bit cache for the tests: values that tell one part of a sequence from another, and a bound on
the decode's error that stays far below what losing a part of the sequence changes."""
import math

import torch

import q4_reference as R


def rows(hkv, spread=0.0):
    """K and V of n tokens: N(0, 1), every 256 tokens of V around levels of their own (N(0, 2), one for each head and group
    of 32 dims). With `spread`, every 2048 keys are longer or shorter by e^N(0, spread), so that chunks have maxima of their own."""
    def make(n, gen):
        dev = gen.device
        k, v = (torch.randn((n, hkv, 128), generator=gen, device=dev) for _ in range(2))
        level = 2.0 * torch.randn((-(-n // 256), hkv, 4), generator=gen, device=dev).repeat_interleave(32, 2)
        size = torch.exp(spread * torch.randn((-(-n // 2048), 1, 1), generator=gen, device=dev))
        return k * size.repeat_interleave(2048, 0)[:n], v + level.repeat_interleave(256, 0)[:n]
    return make


def weights(q, k, scale):
    """Softmax weights [hq, n] of one query [1, hq, 128] over keys [n, hkv, 128], in 64 bits."""
    s = torch.einsum("hd,thd->ht", q[0].double(), k.double().repeat_interleave(q.shape[1] // k.shape[1], 1)) * scale
    return torch.softmax(s, -1)


def tolerance(ref, q, k, v, s_v, scale):
    """A bound on the decode's error for one query, [hq, 128], from the same values that `ref` was computed of.

    A token's p s is rounded to fp16 times a power of two: off by b = 2^-11 p s where that is a normal number, and by no
    more than min(2^-25 P, p s) where it is subnormal, P being the largest p s of the tokens, groups and heads that share
    the power (here: of all the query's). A code multiplies it by at most 15. The roundings of different tokens are
    independent, so by Hoeffding's inequality their sum passes 8 sqrt(sum (15 b)^2) with a probability of 2 e^-32.
    Logits are fp32 sums of 128 products, off by at most 2^-20 of the sum A of their magnitudes, which moves p and the
    sum of p by that much each; the exponential and the remaining fp32 sums: 2^-20 of the values. The result is rounded
    once, by half a step."""
    half = torch.finfo(q.dtype).eps / 2
    g = q.shape[1] // k.shape[1]
    w = weights(q, k, scale)
    ws = w[..., None] * s_v.double().transpose(0, 1).repeat_interleave(g, 0)             # [hq, n, 4]
    b = 15 * torch.maximum(ws * 2.0 ** -11, ws.clamp(max=2.0 ** -25 * float(ws.max())))
    rounding = 8 * b.square().sum(1).sqrt()                                              # [hq, 4]
    size = v.double().unflatten(-1, (4, 32)).abs().amax((0, -1)) + 15 * s_v.double().amax(0)
    a = (torch.einsum("hd,thd->ht", q[0].double().abs(), k.double().abs().repeat_interleave(g, 1)) * scale).amax(1)
    fp32 = size.repeat_interleave(g, 0) * 2.0 ** -20 * (1 + 2 * a[:, None])
    t = (rounding + fp32).repeat_interleave(32, -1)
    return half * (ref.abs() + t) + t + 2.0 ** -25


def reference(q, k_rows, v_rows, scale):
    """(result, bound) of one query [1, hq, 128] over stored rows [n, hkv, 128] of the call's type."""
    k = R.dequantised(k_rows)
    cv, sv, zv = R.quantise(v_rows)
    v = R.values(cv, sv, zv)
    ref = R.attention(q, k, v, k.shape[0] - 1, scale)[0]
    tol = tolerance(ref, q, k, v, sv, scale)
    assert float(tol.max()) <= 0.05 * float(ref.abs().max()), "the bound has to be far below the result"
    return ref, tol


def as_the_kernel_rounds(q, k_rows, v_rows, scale, chunk, lost=(), off=()):
    """The decode's own steps in 64 bits but for p s, rounded to fp16 after a power of two for each 64 tokens. Chunks in
    `lost` are left out; those in `off` are joined with half their weight."""
    k = R.dequantised(k_rows)
    cv, sv, zv = R.quantise(v_rows)
    g = q.shape[1] // k.shape[1]
    w = weights(q, k, scale)
    n = w.shape[1]
    num = torch.zeros((q.shape[1], 128), dtype=torch.float64)
    den = torch.zeros((q.shape[1], 1), dtype=torch.float64)
    for i, c0 in enumerate(range(0, n, chunk)):
        if i in lost:
            continue
        f = 0.5 if i in off else 1.0
        for a in range(c0, min(n, c0 + chunk), 64):
            e = min(n, c0 + chunk, a + 64)
            p = w[:, a:e, None]
            ps = p * sv[a:e].double().transpose(0, 1).repeat_interleave(g, 0)
            power = 2.0 ** -math.floor(math.log2(max(float(ps.max()), 1e-300)))
            ps = (ps * power).to(torch.float16).double() / power
            codes = cv[a:e].double().transpose(0, 1).repeat_interleave(g, 0)
            z = zv[a:e].double().transpose(0, 1).repeat_interleave(g, 0)
            num += f * ((ps.repeat_interleave(32, -1) * codes).sum(1) + (p * z).sum(1).repeat_interleave(32, -1))
            den += f * p.sum(1)
    return (num / den).to(q.dtype).double()
