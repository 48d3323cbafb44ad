"""Prefill with modified scores where the scores are large, against the 64-bit definition: a row's shares depend on what
its scores differ by, whatever their size."""
import pytest
import torch

import mods_reference as R

pytestmark = pytest.mark.gpu
D, BS = 128, 256


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


def _exact_rows(cached, new, hq, hkv, dtype, sizes, sign, seed=1):
    """q, k whose products are whole multiples of 1/4 below 2^17, so that 32 bits hold them exactly: dims 0 and 1 only.
    Row i's largest scores are about sign * sizes[i % len(sizes)], at some keys, a few units apart; at the others they are
    lower by a sixteenth of that at least."""
    g = torch.Generator().manual_seed(seed)
    total = cached + new
    q, k = torch.zeros((new, hq, D)), torch.zeros((total, hkv, D))
    a = torch.tensor([sizes[i % len(sizes)] for i in range(new)]) / 64.0
    q[:, :, 0] = a.to(dtype).float()[:, None]                       # 8 bits at most in the smaller type: a * 64 is exact
    q[:, :, 1] = 1.0
    high, low = (64.0, 60.0) if sign > 0 else (-60.0, -64.0)
    some = torch.rand((total, hkv), generator=g) < 0.1
    some[0] = True                                                  # every row sees one
    k[:, :, 0] = torch.where(some, high, low)
    k[:, :, 1] = torch.randint(-12, 13, (total, hkv), generator=g) / 4.0
    v = torch.randn((total, hkv, D), generator=g)
    return q.to(dtype).cuda(), k.to(dtype).cuda(), v.to(dtype).cuda()


def _check(out, q, k, v, cached, dtype, scale=1.0, **mods):
    """As exact products leave: z in 32 bits (largest |score| times 2^-24 in each of four steps) makes a share wrong by
    twice what a score is, p rounded to 16 bits, the result's own rounding (as in the tests of ordinary scores)."""
    hq, hkv = q.shape[1], k.shape[1]
    eps = torch.finfo(dtype).eps / 2
    for a in range(0, q.shape[0], 256):
        rows = q[a:a + 256]
        ref, p, _, _ = R.attention_rows(rows, k, v, cached + a, scale, **mods)
        size = torch.einsum("hnt,thd->nhd", p, v.double().abs().repeat_interleave(hq // hkv, 1))
        largest = float(torch.einsum("nhd,thd->hnt", rows.double().abs(),
                                     k.double().abs().repeat_interleave(hq // hkv, 1)).max()) * scale
        if mods.get("slopes") is not None:
            largest += float(mods["slopes"].abs().max()) * k.shape[0]
        off = largest * 2.0 ** -22 + 2.0 ** -18
        room = ref.abs() * 2 * eps + size * (eps + 2 * off) + 2.0 ** -25
        err = (out[a:a + 256].double() - ref).abs()
        assert bool((err <= room).all()), (a, float((err / room).max()), float(out[a:a + 256].abs().max()))


def _run(pkv, q, k, v, cached, scale=1.0, **mods):
    fn = pkv.pkv_prefill_varlen_mod_f16 if q.dtype == torch.float16 else pkv.pkv_prefill_varlen_mod
    cu = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (q.shape[0], k.shape[0])]
    return fn(q, *cu, q.shape[0], k.shape[0], scale, k=k, v=v, **mods)


SIZES = [1000.0, 2100.0, 5700.0, 5712.0, 5736.0, 5780.0, 5860.0, 8010.0, 11500.0, 17000.0, 22800.0, 23000.0, 25000.0, 30000.0]


# whole items; items whose keys are split over a cluster; whole rounds of items and a rest
@pytest.mark.parametrize("cached,new,hq,hkv", [(130, 200, 4, 2), (0, 300, 3, 1), (2500, 200, 4, 2), (300, 2600, 16, 8)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_large_scores(pkv, dtype, sign, cached, new, hq, hkv):
    q, k, v = _exact_rows(cached, new, hq, hkv, dtype, SIZES, sign)
    for window in (0, 190):
        _check(_run(pkv, q, k, v, cached, window=window), q, k, v, cached, dtype, window=window)
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("cached,new", [(130, 200), (2500, 200)])
@pytest.mark.parametrize("sign", [1, -1])
def test_larger_scores(pkv, sign, cached, new):
    """bf16 rows, whose shares have fp32's range."""
    q, k, v = _exact_rows(cached, new, 4, 2, torch.bfloat16, [i * 1000.0 + 40.0 * (i % 7) for i in range(30, 64)], sign)
    _check(_run(pkv, q, k, v, cached), q, k, v, cached, torch.bfloat16)
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("cap", [10000.0, 1e6])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_large_scores_under_a_large_cap(pkv, dtype, cap):
    """A cap beyond the scores: rows whose scores are 1000 and 2100, a fifth of the cap at most. Its tanh is off by 6.9e-6
    of a score (bf16), 6.1e-7 (fp16), that of scores a few units apart by as much."""
    q, k, v = _exact_rows(300, 200, 4, 2, dtype, SIZES[:2], 1)
    out = _run(pkv, q, k, v, 300, softcap=cap)
    hq, hkv = 4, 2
    eps = torch.finfo(dtype).eps / 2
    ref, p, _, _ = R.attention_rows(q, k, v, 300, 1.0, softcap=cap)
    size = torch.einsum("hnt,thd->nhd", p, v.double().abs().repeat_interleave(hq // hkv, 1))
    off = 2112 * ((6.9e-6 if dtype == torch.bfloat16 else 6.1e-7) + 2.0 ** -21) + 2.0 ** -18
    room = ref.abs() * 2 * eps + size * (eps + 2 * off) + 2.0 ** -25
    assert bool(((out.double() - ref).abs() <= room).all())


@pytest.mark.parametrize("cached,new", [(900, 130), (8000, 70), (20000, 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_negative_slopes(pkv, dtype, cached, new):
    """A bias that favours far keys: the largest scores are about the distance to the first key."""
    q, k, v = _exact_rows(cached, new, 4, 2, dtype, [4.0], 1)
    slopes = torch.tensor([-1.0, -0.5, -0.25, -1.5], device="cuda")
    _check(_run(pkv, q, k, v, cached, slopes=slopes), q, k, v, cached, dtype, slopes=slopes)
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("cached", [12000, 40000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_bias_far_from_the_keys(pkv, dtype, cached):
    """Usual slopes over long ranges of keys that clusters share: the parts far from the rows have scores of -8000 and below."""
    new, hq, hkv = 64, 16, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn((n, h, D), generator=g, device="cuda").to(dtype)
               for n, h in ((new, hq), (cached + new, hkv), (cached + new, hkv)))
    slopes = torch.tensor([2.0 ** (-0.5 * (h + 1)) for h in range(hq)], device="cuda")
    scale = D ** -0.5
    out = _run(pkv, q, k, v, cached, scale=scale, slopes=slopes)
    eps = torch.finfo(dtype).eps / 2
    for a in range(0, new, 16):
        ref, p, bound, _ = R.attention_rows(q[a:a + 16], k, v, cached + a, scale, slopes=slopes)
        size = torch.einsum("hnt,thd->nhd", p, v.double().abs().repeat_interleave(hq // hkv, 1))
        # shares fall by 2^-24 within 24 / slope keys, 4096 of the flattest head, where the distance term is 16 or less
        room = ref.abs() * 2 * eps + size * (eps + 2.0 ** -16) + bound + 2.0 ** -25
        err = (out[a:a + 16].double() - ref).abs()
        assert bool((err <= room).all()), float((err / room).max())
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("cached,new,hq,hkv", [(300, 150, 4, 2), (0, 300, 3, 1), (3000, 100, 4, 2)])
@pytest.mark.parametrize("gap", [9.0, 12.0, 14.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_shares_far_below_the_largest(pkv, dtype, gap, cached, new, hq, hkv):
    """A first key that takes nearly all of the weight and has nothing to say: the result is the others' small shares, from
    2^-13 to 2^-21 of the largest, each of which is rounded by half a step of 16 bits."""
    total = cached + new
    g = torch.Generator().manual_seed(3)
    q, k = torch.zeros((new, hq, D)), torch.zeros((total, hkv, D))
    q[:, :, 0] = 1.0
    k[:, :, 0] = torch.randint(0, 3, (total, hkv), generator=g) / 4.0
    k[0, :, 0] = gap
    v = torch.rand((total, hkv, D), generator=g) + 0.5
    v[0] = 0
    q, k, v = (x.to(dtype).cuda() for x in (q, k, v))
    _check(_run(pkv, q, k, v, cached), q, k, v, cached, dtype)
    slopes = torch.full((hq,), 2.0 ** -12, device="cuda")
    _check(_run(pkv, q, k, v, cached, slopes=slopes), q, k, v, cached, dtype, slopes=slopes)
