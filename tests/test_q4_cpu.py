"""CPU checks of the 4-bit cache's entry points: arguments refused on the host
before anything is launched, workspace sizes, and the reference's own format."""
import ctypes

import pytest
import torch

import q4_reference as R

ONE = ctypes.c_void_p(16)
ODD = ctypes.c_void_p(24)


@pytest.fixture(scope="module")
def lib():
    import paged_kv_cache_kvh_gb300 as m
    return m._lib


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_store_and_load_refusals(lib, suffix):
    store, load = getattr(lib, "pkv_store_kvcache_q4" + suffix), getattr(lib, "pkv_load_kvcache_q4" + suffix)

    def st(k=ONE, ks=1024, v=ONE, vs=1024, kc=ONE, vc=ONE, sm=ONE, n=4, h=8, d=128, bs=256, nb=2):
        return store(k, ks, v, vs, kc, vc, sm, n, h, d, bs, nb, None)

    def ld(kc=ONE, vc=ONE, sm=ONE, n=4, h=8, d=128, bs=256, nb=2, k=ONE, v=ONE):
        return load(kc, vc, sm, n, h, d, bs, nb, k, v, None)

    for f in (st, ld):
        assert f(d=64) == f(bs=16) == f(h=0) == f(h=-1) == f(h=8193) == -2
        assert f(n=-1) == f(nb=-1) == -6
        assert f(n=0, k=None) == 0
        for name in ("k", "v", "kc", "vc", "sm"):
            assert f(**{name: None}) == -1
        assert f(kc=ODD) == f(vc=ODD) == -4
    assert st(ks=1023) == st(vs=0) == -3
    assert st(k=ctypes.c_void_p(17)) == -4
    assert ld(k=ODD) == ld(v=ODD) == -4


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_decode_refusals(lib, suffix):
    dec, step = getattr(lib, "pkv_decode_q4" + suffix), getattr(lib, "pkv_store_decode_q4" + suffix)
    need = lib.pkv_decode_q4_workspace_bytes(4, 16, 8, 4096)

    def common(q=ONE, qs=2048, kc=ONE, vc=ONE, nb=16, bt=ONE, bs=16, cl=ONE, n=4, hq=16, hkv=8, d=128, blk=256,
               mc=4096, sc=0.1, out=ONE, ws=ONE, wb=need):
        return (q, qs), (kc, vc, nb, bt, bs, cl, n, hq, hkv, d, blk, mc, sc, out, ws, wb, None)

    def d(**kw):
        a, b = common(**kw)
        return dec(*a, *b)

    def s(k=ONE, ks=1024, v=ONE, vs=1024, sm=ONE, **kw):
        a, b = common(**kw)
        return step(*a, k, ks, v, vs, sm, *b)

    for f in (d, s):
        assert f(d=64) == f(blk=16) == f(hq=24, qs=4096) == f(hq=12) == f(hq=40, qs=8192) == f(hkv=0) == -2
        assert f(n=-1) == f(n=65536) == f(nb=-1) == f(bs=-1) == f(mc=-1) == f(mc=(1 << 24) + 1) == -6
        assert f(sc=0.0) == f(sc=-1.0) == f(sc=float("nan")) == -6
        for name in ("q", "kc", "vc", "bt", "cl", "out"):
            assert f(**{name: None}) == -1
        assert f(qs=2047) == -3
        assert f(q=ODD) == f(qs=2052) == f(kc=ODD) == f(vc=ODD) == f(out=ODD) == f(ws=ODD) == -4
        assert f(ws=None) == f(wb=need - 1) == -5
        assert f(n=0, q=None) == 0
    assert s(k=None) == s(v=None) == s(sm=None) == -1
    assert s(ks=1000) == s(vs=1000) == -3
    assert s(k=ODD) == s(v=ODD) == s(ks=1028) == s(vs=1028) == -4


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_prefill_refusals(lib, suffix):
    pre = getattr(lib, "pkv_prefill_varlen_q4" + suffix)

    def f(q=ONE, qs=2048, tq=10, kc=ONE, vc=ONE, nb=4, cq=ONE, ck=ONE, mq=10, mk=10, bt=ONE, bs=2, n=1, hq=16, hkv=8,
          d=128, blk=256, sc=0.1, out=ONE, ws=None, wb=0):
        return pre(q, qs, tq, kc, vc, nb, cq, ck, mq, mk, bt, bs, n, hq, hkv, d, blk, sc, out, ws, wb, None)

    assert f(d=96) == f(blk=16) == f(hq=8) == f(hq=24, qs=4096) == f(hq=40, qs=8192) == f(hkv=0) == -2
    assert f(tq=-1) == f(nb=-1) == f(mq=-1) == f(mk=-1) == f(bs=-1) == f(n=-1) == f(n=65536) == -6
    assert f(sc=0.0) == f(sc=float("nan")) == f(nb=0) == f(bs=0) == -6
    for name in ("q", "kc", "vc", "cq", "ck", "bt", "out"):
        assert f(**{name: None}) == -1
    assert f(qs=2047) == -3
    assert f(q=ODD) == f(qs=2052) == f(kc=ODD) == f(vc=ODD) == f(out=ODD) == f(ws=ctypes.c_void_p(18), wb=4) == -4
    assert f(ws=ONE, wb=6) == -6
    assert f(n=0, q=None) == f(tq=0, q=None) == f(mq=0, q=None) == 0


def test_workspace_sizes(lib):
    f = lib.pkv_decode_q4_workspace_bytes
    assert f(0, 16, 8, 4096) == f(4, 24, 8, 4096) == f(4, 16, 8, -1) == f(65536, 16, 8, 10) == f(1, 3, 2, 10) == 0
    assert f(1, 16, 8, 0) > 0
    for hq in (8, 16, 32):
        sizes = [f(n, hq, 8, c) for n, c in ((1, 32), (4, 511), (256, 4096), (512, 4096), (1024, 4096))]
        assert sizes == sorted(sizes) and sizes[0] >= 8 * (hq // 8) * 520
    # launches of 768 sequences share it
    assert f(5000, 16, 8, 4096) == f(768, 16, 8, 4096)


def test_workspace_covers_every_slot():
    """The slots for partial results that the chunk rule makes of any context lengths stay within the workspace's
    bound (both restated here), and the tickets within their share of the bytes."""
    import random
    def chunk(halves, units, plan):
        if halves <= plan:
            return 32
        x = -(-units // plan)
        return 64 * -(-x // -(-x // 32))

    def bound(n, rows, ctx, plan):
        units, halves = n * -(-ctx // 64) * rows, n * (ctx // 32) * rows
        return min(halves, max(256 * plan // 17 + 1, units // 29 + 1)) + n * rows

    rng = random.Random(1)
    for _ in range(4000):
        n, hkv = rng.choice([1, 2, 7, 64, 300, 768]), rng.choice([1, 2, 5, 8, 40])
        ctx = int(2 ** rng.uniform(0, 17))
        lens = [rng.randint(0, ctx) if rng.random() < 0.8 else ctx for _ in range(n)]
        for group in (1, 2, 4):
            plan, rows = 152 * 12, hkv * max(1, group // 2)
            c = chunk(sum(-(-x // 32) for x in lens) * rows, sum(-(-x // 64) for x in lens) * rows, plan)
            assert c == 32 or (c % 64 == 0 and c <= 2048)
            m, heads = bound(n, rows, ctx, plan), min(group, 2)
            assert sum(x // c for x in lens) * rows + n * rows <= m
            assert max(-(-x // c) for x in lens) < 2 ** 15
            size = ((m * heads * 520 + 512) // 127 * 128 + 512 + 255) // 256 * 256
            counters = 256 + (size // 128 & ~255)
            assert 8 + 4 * m <= counters and counters + m * heads * 520 <= size


def test_reference_places_are_a_permutation():
    for is_v in (False, True):
        seen = {R.code_place(d, t, is_v) for t in range(16) for d in range(128)}
        assert len(seen) == 2048 and {at for at, _ in seen} == set(range(1024))


def test_reference_quantiser():
    x = torch.linspace(-2, 2, 128, dtype=torch.float64)
    code, s, z = R.quantise(x)
    err = (R.values(code, s, z) - x).abs().unflatten(0, (4, 32))
    assert bool((err <= s.double()[:, None] * 0.5 + 2.0 ** -9).all())
    assert int(code.min()) == 0 and int(code.max()) == 15
