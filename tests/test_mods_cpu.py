"""CPU checks of attention with modified scores: arguments refused on the host, workspace sizes."""
import ctypes

import pytest

ONE = ctypes.c_void_p(16)
ODD = ctypes.c_void_p(24)


@pytest.fixture(scope="module")
def lib():
    import paged_kv_cache_kvh_gb300 as m
    return m._lib


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_decode_refusals(lib, suffix):
    dec = getattr(lib, "pkv_decode_mod" + suffix)
    need = lib.pkv_decode_mod_workspace_bytes(4, 16, 8, 4096, 0)
    more = lib.pkv_decode_mod_workspace_bytes(4, 16, 8, 4096, 1)
    assert more > need > 0

    def f(q=ONE, qs=2048, kc=ONE, vc=ONE, nb=16, bt=ONE, bs=16, cl=ONE, n=4, hq=16, hkv=8, d=128, blk=256, mc=4096, sc=0.1,
          cap=0.0, sl=None, win=0, st=None, w=None, out=ONE, ws=ONE, wb=need):
        return dec(q, qs, kc, vc, nb, bt, bs, cl, n, hq, hkv, d, blk, mc, sc, cap, sl, win, st, w, out, ws, wb, None)

    assert f(d=64) == f(blk=16) == f(hq=12) == f(hkv=0) == f(hq=0) == f(hq=-8) == f(hq=8200, qs=1 << 21) == -2
    assert f(n=-1) == f(n=65536) == f(nb=-1) == f(nb=0) == f(nb=1 << 23) == f(bs=-1) == f(mc=-1) == f(mc=(1 << 24) + 1) == -6
    assert f(sc=0.0) == f(sc=float("nan")) == f(sc=float("inf")) == f(cap=-1.0) == f(cap=float("nan")) == -6
    assert f(cap=float("inf")) == f(win=-1) == -6
    for name in ("q", "kc", "vc", "bt", "cl", "out"):
        assert f(**{name: None}) == -1
    assert f(qs=2047) == -3
    assert f(q=ODD) == f(qs=2052) == f(kc=ODD) == f(vc=ODD) == f(out=ODD) == f(ws=ODD) == -4
    for name in ("sl", "st", "w"):
        assert f(**{name: ctypes.c_void_p(18), "wb": more}) == -4
    assert f(ws=None) == f(wb=need - 1) == f(w=ONE, wb=more - 1) == -5
    assert f(n=0, q=None) == 0


def test_decode_workspace_sizes(lib):
    size = lib.pkv_decode_mod_workspace_bytes
    assert size(0, 16, 8, 4096, 0) == size(65536, 16, 8, 4096, 0) == size(4, 12, 8, 4096, 0) == size(4, 16, 8, -1, 0) == 0
    # partial results: bounded by the GPU's workers, whatever the batch; scores: one per (sequence, token, head)
    assert size(65535, 16, 8, 1 << 24, 0) == size(1, 16, 8, 16, 0) < 1 << 26
    assert size(256, 16, 8, 4096, 1) >= 256 * 16 * 4096 * 4


def test_evict_refusals(lib):
    def f(kc=ONE, vc=ONE, w=ONE, nb=16, bt=ONE, bs=16, cl=ONE, n=4, h=8, d=128, blk=256, mc=4096, budget=300, first=4,
          recent=32, nt=ONE, ns=2, kept=ONE, nl=ONE):
        return lib.pkv_evict_kvcache(kc, vc, w, nb, bt, bs, cl, n, h, d, blk, mc, budget, first, recent, nt, ns, kept, nl,
                                     None)

    assert f(d=64) == f(blk=16) == f(h=0) == f(h=8193) == -2
    assert f(n=-1) == f(n=65536) == f(nb=-1) == f(bs=-1) == f(mc=-1) == f(mc=(1 << 24) + 1) == -6
    assert f(budget=0) == f(budget=(1 << 24) + 1) == f(first=-1) == f(recent=-1) == f(first=301) == f(recent=297) == -6
    assert f(first=(1 << 31) - 1, recent=(1 << 31) - 1) == f(ns=1) == f(ns=-1) == -6
    for name in ("kc", "vc", "w", "bt", "cl", "kept", "nl"):
        assert f(**{name: None}) == -1
    assert f(kc=ODD) == f(vc=ODD) == -4
    for name in ("w", "bt", "cl", "nt", "kept", "nl"):
        assert f(**{name: ctypes.c_void_p(18)}) == -4
    assert f(n=0, kc=None) == 0


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_prefill_refusals(lib, suffix):
    pre = getattr(lib, "pkv_prefill_varlen_mod" + suffix)

    def f(q=ONE, qs=2048, tq=10, k=None, v=None, ks=0, tk=0, kc=ONE, vc=ONE, nb=4, cq=ONE, ck=ONE, mq=10, mk=10, bt=ONE,
          bs=2, n=1, hq=16, hkv=8, d=128, blk=256, sc=0.1, cap=0.0, sl=None, win=0, st=None, pl=None, out=ONE):
        return pre(q, qs, tq, k, v, ks, tk, kc, vc, nb, cq, ck, mq, mk, bt, bs, n, hq, hkv, d, blk, sc, cap, sl, win, st, pl,
                   out, None)

    flat = dict(bt=None, kc=None, vc=None, k=ONE, v=ONE, ks=1024, tk=10)
    assert f(d=64) == f(blk=16) == f(hq=12) == f(hkv=0) == f(hq=8200, hkv=8200) == -2
    for name in ("n", "tq", "tk", "mq", "mk", "win"):
        assert f(**{name: -1}) == -6
    assert f(n=65536) == f(mq=(1 << 24) + 1) == f(mk=(1 << 24) + 1) == f(nb=0) == f(nb=1 << 23) == f(bs=0) == -6
    assert f(**{**flat, "tk": 0}) == f(sc=0.0) == f(sc=float("inf")) == f(cap=-1.0) == f(cap=float("nan")) == -6
    for name in ("q", "out", "cq", "ck", "kc", "vc"):
        assert f(**{name: None}) == -1
    assert f(**{**flat, "k": None}) == f(**{**flat, "v": None}) == -1
    assert f(qs=2047) == f(**{**flat, "ks": 1023}) == -3
    assert f(q=ODD) == f(qs=2052) == f(out=ODD) == f(kc=ODD) == f(vc=ODD) == f(**{**flat, "ks": 1028}) == -4
    for name in ("sl", "st", "pl"):
        assert f(**{name: ctypes.c_void_p(18)}) == -4
    assert f(n=0, q=None) == f(tq=0, q=None) == f(mq=0, q=None) == 0
