"""CPU checks of the rotary positions' entry points: frequencies against their formulas, arguments refused on the host."""
import ctypes
import math

import numpy as np
import pytest

ONE = ctypes.c_void_p(16)
ODD = ctypes.c_void_p(17)


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_kvh_gb300 as m
    return m


def _formula(rot, theta, scaling, factor, orig, a, b):
    if scaling == "ntk" and rot > 2:
        theta = theta * factor ** (rot / (rot - 2))
    out = []
    if scaling == "yarn":
        def place(turns):
            return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(theta))
        low, high = max(math.floor(place(a)), 0), min(math.ceil(place(b)), rot - 1)
    for i in range(rot // 2):
        f = theta ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "bands":
            g = min(1, max(0, (orig * f / (2 * math.pi) - a) / (b - a)))
            f = g * f + (1 - g) * f / factor
        if scaling == "yarn":
            g = min(1, max(0, (i - low) / max(high - low, 1e-3)))
            f = (1 - g) * f + g * f / factor
        out.append(f)
    return out


@pytest.mark.parametrize("rot", [2, 6, 64, 96, 128, 1024])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "bands", "yarn"])
def test_frequencies(pkv, rot, scaling):
    for theta, factor, orig in ((1e6, 4.0, 32768), (1e4, 8.5, 4096), (5e5, 1.0, 8192)):
        ramp = (32.0, 1.0) if scaling == "yarn" else (1.0, 4.0)
        got, mag = pkv.rope_frequencies(rot, theta, scaling, factor=factor, original_max_position=orig, ramp=ramp,
                                        device=None)
        want = _formula(rot, theta, scaling, factor, orig, *ramp)
        assert got.dtype == np.int64 and got.shape == (rot // 2,)
        # 64-bit powers and products: a few steps of 2^-53 each, the exponent's error times ln(theta) < 14
        for x, w in zip(got.tolist(), want):
            assert abs(x - w / (2 * math.pi) * 2.0 ** 64) <= w / (2 * math.pi) * 2.0 ** 64 * 2.0 ** -40 + 1
        assert mag == pytest.approx(0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0, rel=2.0 ** -23)


def test_frequencies_refusals(pkv):
    f = pkv._lib.pkv_rope_frequencies
    out, mag = (ctypes.c_int64 * 64)(), ctypes.c_float()
    def call(r=128, theta=1e6, sc=0, factor=1.0, orig=4096.0, a=1.0, b=4.0, o=out, m=ctypes.addressof(mag)):
        return f(r, theta, sc, factor, orig, a, b, o, m)
    assert call() == 0
    assert call(o=None) == call(m=None) == -1
    assert call(r=0) == call(r=3) == call(r=1026) == call(r=-2) == call(sc=-1) == call(sc=5) == -2
    assert call(theta=1.0) == call(theta=float("nan")) == call(theta=float("inf")) == -6
    assert call(sc=1, factor=0.5) == call(sc=1, factor=float("inf")) == call(sc=1, factor=float("nan")) == -6
    assert call(sc=3, orig=0.0) == call(sc=3, a=4.0, b=4.0) == call(sc=3, a=float("nan")) == -6
    assert call(sc=4, a=1.0, b=32.0) == call(sc=4, a=32.0, b=0.0) == -6
    assert call(sc=4, a=32.0, b=1.0) == call(sc=3, factor=2.0) == 0
    assert call(factor=0.0) == 0          # not used without a scaling
    for kw in (dict(scaling="other"), dict(rotary_dim=0), dict(rotary_dim=-4)):
        with pytest.raises(ValueError):
            pkv.rope_frequencies(device=None, **kw)
    with pytest.raises(pkv.PkvError):
        pkv.rope_frequencies(7, device=None)


@pytest.mark.parametrize("suffix", ["", "_f16"])
def test_refusals(pkv, suffix):
    rope, store = getattr(pkv._lib, "pkv_rope" + suffix), getattr(pkv._lib, "pkv_rope_store_kvcache" + suffix)

    def alone(q=ONE, qs=2048, k=ONE, ks=1024, pos=ONE, fr=ONE, r=128, mag=1.0, il=0, n=4, hq=16, hkv=8, d=128, qo=ONE,
              qos=2048, ko=ONE, kos=1024):
        return rope(q, qs, k, ks, pos, fr, r, mag, il, n, hq, hkv, d, qo, qos, ko, kos, None)

    def both(q=ONE, qs=2048, k=ONE, ks=1024, v=ONE, vs=1024, pos=ONE, fr=ONE, r=128, mag=1.0, il=0, sm=ONE, n=4, hq=16,
             hkv=8, d=128, ns=512, qo=ONE, qos=2048, kc=ONE, vc=ONE):
        return store(q, qs, k, ks, v, vs, pos, fr, r, mag, il, sm, n, hq, hkv, d, ns, qo, qos, kc, vc, None)

    for f in (alone, both):
        assert f(r=0) == f(r=127) == f(r=130) == f(d=0) == f(d=1026) == f(hq=-1) == f(hkv=-1) == f(hq=8193) == -2
        assert f(n=-1) == f(mag=float("nan")) == f(mag=float("inf")) == -6
        assert f(n=0, q=None, k=None, pos=None) == f(hq=0, hkv=0, q=None, k=None) == 0
        for name in ("q", "k", "pos", "fr", "qo"):
            assert f(**{name: None}) == -1
        assert f(qs=2047) == f(ks=1023) == f(qos=2047) == -3
        assert f(q=ODD) == f(k=ODD) == f(qo=ODD) == f(pos=ctypes.c_void_p(20)) == f(fr=ctypes.c_void_p(12)) == -4
    assert alone(ko=None) == both(v=None) == both(kc=None) == both(vc=None) == both(sm=None) == -1
    assert alone(kos=1023) == both(vs=1023) == -3
    assert alone(ko=ODD) == both(kc=ODD) == both(v=ODD) == both(sm=ctypes.c_void_p(18)) == -4
    assert both(ns=-1) == -6
