"""Decode with modified scores over values that are not finite: NaN and infinities of keys that take part come out as the
definition has them, with partial results joined, and those of other keys reach nothing."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D, BS = 128, 256


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


def _by_definition(q, k, v, lo, window, softcap):
    """One row [hq, D] over keys [n, hkv, D] in 64 bits, from the keys that it sees and no others."""
    hq, n, hkv = q.shape[0], k.shape[0], k.shape[1]
    lo = max(lo, n - window if window else 0)
    out = torch.zeros((hq, D), dtype=torch.float64)
    if lo >= n:
        return out
    for h in range(hq):
        s = k[lo:, h // (hq // hkv)].double() @ q[h].double() * D ** -0.5
        s = softcap * torch.tanh(s / softcap) if softcap else s
        e = torch.exp(s - s.max())
        out[h] = (e[:, None] / e.sum() * v[lo:, h // (hq // hkv)].double()).sum(0)
    return out


@pytest.mark.parametrize("mods", [{}, dict(window=90), dict(starts=True), dict(softcap=10.0)])
@pytest.mark.parametrize("hq,hkv", [(16, 8), (12, 1), (3, 3)])
@pytest.mark.parametrize("lens", [[100, 1, 31, 300, 17], [6000], [2000, 90, 2500]])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_what_is_not_finite(pkv, dtype, lens, hq, hkv, mods):
    g = torch.Generator(device="cuda").manual_seed(len(lens) + hq)
    cpu = torch.Generator().manual_seed(5)
    per = [-(-n // BS) for n in lens]
    ids = iter(range(sum(per)))
    tables = [[next(ids) for _ in range(m)] + [0] * (max(per) - m) for m in per]
    kc, vc = (torch.randn((sum(per), BS, hkv, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((len(lens), hq, D), generator=g, device="cuda").to(dtype)
    odd = [float("nan"), float("inf"), float("-inf")]
    for _ in range(60):
        b = int(torch.randint(0, len(lens), (1,), generator=cpu))
        t, h, d = (int(torch.randint(0, m, (1,), generator=cpu)) for m in (lens[b], hkv, 16))
        vc[tables[b][t // BS], t % BS, h, d] = odd[int(torch.randint(0, 3, (1,), generator=cpu))]
    starts = [n // 3 for n in lens] if mods.get("starts") else [0] * len(lens)
    asked = {name: mods[name] for name in ("window", "softcap") if name in mods}
    if mods.get("starts"):
        asked["key_starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    call = pkv.pkv_decode_mod_f16 if dtype == torch.float16 else pkv.pkv_decode_mod
    for weights in (None, pkv.attention_weights(sum(per), hkv)):
        ws = pkv.decode_mod_workspace(len(lens), max(lens), hq, hkv, weights=weights is not None)
        out = call(q, kc, vc, torch.tensor(tables, dtype=torch.int32, device="cuda"),
                   torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens), D ** -0.5, ws, weights=weights, **asked)
        assert pkv.pkv_device_error() == 0
        if weights is not None:
            assert bool(torch.isfinite(weights).all())     # shares come from scores alone
        eps = torch.finfo(dtype).eps / 2
        for b, n in enumerate(lens):
            blocks = torch.tensor(tables[b][:per[b]], device="cuda")
            k, v = (c[blocks].flatten(0, 1)[:n].cpu() for c in (kc, vc))
            ref = _by_definition(q[b].cpu(), k, v, starts[b], mods.get("window", 0), mods.get("softcap", 0.0))
            got = out[b].double().cpu()
            assert torch.equal(torch.isnan(got), torch.isnan(ref))
            inf = torch.isinf(ref)
            assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], ref[inf])
            fine = torch.isfinite(ref)
            largest = float(torch.where(torch.isfinite(v), v, torch.zeros_like(v)).double().abs().max())
            # the result's rounding, and 2^-15 of sum p |v|: p in two parts, scores of a few units in 32 bits
            assert bool(((got - ref).abs() <= eps * ref.abs() + 2.0 ** -15 * largest)[fine].all())


@pytest.mark.parametrize("gap", [9.0, 12.0, 14.0])
@pytest.mark.parametrize("hq,hkv,n", [(16, 8, 700), (12, 1, 5000), (2, 1, 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_shares_far_below_the_largest(pkv, dtype, hq, hkv, n, gap):
    """A first key that takes nearly all of the weight and whose value is nothing: the result is the others' small shares."""
    g = torch.Generator().manual_seed(3)
    blocks = -(-n // BS)
    q, kc, vc = torch.zeros((1, hq, D)), torch.zeros((blocks, BS, hkv, D)), torch.rand((blocks, BS, hkv, D), generator=g) + 0.5
    q[..., 0] = 1.0
    kc[..., 0] = torch.randint(0, 3, (blocks, BS, hkv), generator=g) / 4.0
    kc[0, 0, :, 0] = gap
    vc[0, 0] = 0
    q, kc, vc = (x.to(dtype).cuda() for x in (q, kc, vc))
    call = pkv.pkv_decode_mod_f16 if dtype == torch.float16 else pkv.pkv_decode_mod
    out = call(q, kc, vc, torch.arange(blocks, dtype=torch.int32, device="cuda")[None],
               torch.tensor([n], dtype=torch.int32, device="cuda"), n, 1.0, pkv.decode_mod_workspace(1, n, hq, hkv))
    k, v = (c.flatten(0, 1)[:n].cpu() for c in (kc, vc))
    ref = _by_definition(q[0].cpu(), k.double() * D ** 0.5, v, 0, 0, 0.0)
    # the result's rounding; p in two parts (2^-15), scores of 14 units in 32 bits (2^-18)
    room = ref.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -14) + 2.0 ** -25
    assert bool(((out[0].double().cpu() - ref).abs() <= room).all())
