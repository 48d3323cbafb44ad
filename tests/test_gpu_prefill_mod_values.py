"""Prefill with modified scores over values that are not finite and long ranges of keys: they reach the rows that see their
key, in their dim, and nothing else is lost by them."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


def _rows(seqs, hq, hkv, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lq, lk = sum(n for _, n in seqs), sum(c + n for c, n in seqs)
    return [torch.randn((n, h, D), generator=g, device="cuda").to(dtype) for n, h in ((lq, hq), (lk, hkv), (lk, hkv))]


def _run(pkv, q, k, v, seqs, **mods):
    fn = pkv.pkv_prefill_varlen_mod_f16 if q.dtype == torch.float16 else pkv.pkv_prefill_varlen_mod
    cu_q, cu_k = [0], [0]
    for c, n in seqs:
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + c + n)
    cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu_q, cu_k)]
    return fn(q, *cu, max(n for _, n in seqs), max(c + n for c, n in seqs), D ** -0.5, k=k, v=v, **mods)


def _near(a, b, v, where):
    """Rows that are computed again do not round p: half a step of 16 bits of sum p |v| apart, and either result rounded."""
    eps = torch.finfo(a.dtype).eps
    room = eps * (b.float().abs() + float(v.float().abs().nan_to_num(0, 0, 0).max()))
    return bool(((a.float() - b.float()).abs() <= room)[where].all())


@pytest.mark.parametrize("dtype,value", [(torch.bfloat16, float("nan")), (torch.float16, float("inf"))])
def test_one_bad_value_before_a_long_range(pkv, dtype, value):
    """Whole items and split ones, and another sequence behind them. Rows of the first and of the last tile do not see a
    value that their tile's products take in."""
    cached, new = 45000, 12800
    seqs = [(cached, new), (0, 200)]
    q, k, v = _rows(seqs, 2, 1, dtype)
    clean = _run(pkv, q, k, v, seqs)
    v[cached + 127, 0, 5] = value
    v[cached + new - 1, 0, 77] = value
    out = _run(pkv, q, k, v, seqs)
    assert pkv.pkv_device_error() == 0
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[127:new, :, 5] = True
    bad[new - 1, :, 77] = True
    assert torch.equal(~torch.isfinite(out), bad)
    assert _near(out, clean, v, ~bad)


def test_rows_computed_again_for_longer_than_a_wait(pkv):
    """The rows of the first items do not see the last value, which takes one warp more than two seconds to put right; the
    CTA's other roles, which have taken further items meanwhile, wait for it."""
    cached, new, hq = 100000, 12800, 8
    q, k, v = _rows([(cached, new)], hq, 1, torch.bfloat16)
    clean = _run(pkv, q, k, v, [(cached, new)])
    v[cached + new - 1, 0, 77] = float("nan")
    out = _run(pkv, q, k, v, [(cached, new)])
    assert pkv.pkv_device_error() == 0
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[new - 1, :, 77] = True
    assert torch.equal(torch.isnan(out), bad)
    assert _near(out, clean, v, ~bad)


def _by_definition(q, k, v, cached, rows, window=0, starts=None, prefix=0, softcap=0.0):
    """Rows of one sequence in 64 bits, each from the keys that it sees and no others."""
    hq, hkv = q.shape[1], k.shape[1]
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    out = torch.zeros((len(rows), hq, D), dtype=torch.float64)
    for j, i in enumerate(rows):
        p = cached + i
        lo = max(p - window + 1 if window else 0, 0 if starts is None else int(starts[i]))
        hi = min(k.shape[0], max(p + 1, prefix))
        if lo >= hi:
            continue
        for h in range(hq):
            s = k[lo:hi, h // (hq // hkv)] @ q[i, h] * D ** -0.5
            s = softcap * torch.tanh(s / softcap) if softcap else s
            e = torch.exp(s - s.max())
            out[j, h] = (e[:, None] / e.sum() * v[lo:hi, h // (hq // hkv)]).sum(0)
    return out


def _same(out, ref, v):
    """NaN and infinities alike; elsewhere p's rounding to 16 bits (half a step of sum p |v|) and the result's own, and what
    32 bits lose of scores of a few units (2^-16 of sum p |v|)."""
    eps = torch.finfo(out.dtype).eps / 2
    out = out.double().cpu()
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    odd = torch.isinf(ref)
    assert torch.equal(torch.isinf(out), odd) and torch.equal(out[odd], ref[odd])
    fine = torch.isfinite(ref)
    largest = float(torch.where(torch.isfinite(v), v, torch.zeros_like(v)).double().abs().max())
    assert bool(((out - ref).abs() <= 2 * eps * ref.abs() + (eps + 2.0 ** -16) * largest)[fine].all())


KINDS = {
    "plain": {}, "window": dict(window=90), "docs": dict(starts=True), "prefix": dict(prefix=350), "cap": dict(softcap=20.0),
}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("cached,new,hq,hkv", [(300, 280, 4, 2), (0, 300, 3, 1), (2500, 140, 2, 1)])
@pytest.mark.parametrize("where", ["few", "many", "dims", "all"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_what_is_not_finite_row_by_row(pkv, dtype, where, cached, new, hq, hkv, kind):
    """Whole items and split ones. Infinities beside NaN that a row does not see, in the same dim, stay infinities."""
    total = cached + new
    q, k, v = _rows([(cached, new)], hq, hkv, dtype, seed=len(where) + new)
    g = torch.Generator().manual_seed(7)
    odd = [float("nan"), float("inf"), float("-inf")]
    if where in ("few", "many"):
        for _ in range(12 if where == "few" else 400):
            t, h, d = (int(torch.randint(0, n, (1,), generator=g)) for n in (total, hkv, D))
            if where == "few":
                t, d = max(0, total - 1 - t % 260), d % 8          # in the rows' own tiles, and in few dims
            v[t, h, d] = odd[int(torch.randint(0, 3, (1,), generator=g))]
    elif where == "dims":
        v[:, 0, :50] = float("nan")
        v[::7, 0, 60:70] = float("inf")
        v[3::11, 0, 70:75] = float("-inf")
    else:
        v[:] = float("nan")
    mods, asked = dict(KINDS[kind]), {}
    if mods.get("starts"):
        mods["starts"] = torch.tensor([max(0, (cached + i) // 97 * 97) for i in range(new)], dtype=torch.int32)
        mods["starts"][5] = 10 ** 8                                # a row that sees nothing
        asked["key_starts"] = mods["starts"].cuda()
    if mods.get("prefix"):
        mods["prefix"] = min(mods["prefix"] + cached // 2, total)
        asked["prefix_lens"] = torch.tensor([mods["prefix"]], dtype=torch.int32, device="cuda")
    asked.update({n: mods[n] for n in ("window", "softcap") if n in mods})
    out = _run(pkv, q, k, v, [(cached, new)], **asked)
    assert pkv.pkv_device_error() == 0
    rows = sorted(set(range(0, new, 9)) | set(range(120, min(new, 136))) | {0, 1, 5, new - 2, new - 1})
    _same(out[rows], _by_definition(q, k, v, cached, rows, **mods), v)


@pytest.mark.parametrize("cached,new", [(100, 300), (2500, 100)])
def test_sums_beyond_32_bits(pkv, cached, new):
    """Values of up to 3e38 whose weighted mean is finite, beside NaN that some rows see. Scores at a cap of 50 or less take
    no maximum (2^72 of 3e38 is beyond fp32), others one that lags by up to 2^8."""
    q, k, v = _rows([(cached, new)], 4, 2, torch.bfloat16)
    q, k = q.abs() * 3, k.abs()
    v *= 2.0 ** 120
    v[cached + 50, 1, 3] = float("nan")
    rows = list(range(0, new, 7))
    for cap in (0.0, 40.0):
        out = _run(pkv, q, k, v, [(cached, new)], softcap=cap)
        _same(out[rows], _by_definition(q, k, v, cached, rows, softcap=cap), v)
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("hq,hkv", [(2, 1), (3, 1)])
@pytest.mark.parametrize("kind", ["key", "query"])
def test_scores_that_are_not_finite(pkv, kind, hq, hkv):
    """A NaN in a key or a query makes its rows NaN throughout, and no others; many rows of a long range among them."""
    cached, new = 9000, 8000
    q, k, v = _rows([(cached, new)], hq, hkv, torch.bfloat16)
    clean = _run(pkv, q, k, v, [(cached, new)])
    bad = torch.zeros_like(clean, dtype=torch.bool)
    if kind == "key":
        k[cached + 70, 0, 9] = float("nan")
        bad[70:] = True
    else:
        q[1000, 1, 3] = float("nan")
        bad[1000, 1] = True
    out = _run(pkv, q, k, v, [(cached, new)])
    assert torch.equal(torch.isnan(out), bad) and torch.equal(out[~bad], clean[~bad])
    assert pkv.pkv_device_error() == 0
