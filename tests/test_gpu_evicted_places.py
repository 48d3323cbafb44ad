"""What window, slopes and first keys of the decode mean over a cache that has been cut down: places in the cache, head by
head, as documented."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["cap", "window", "slopes", "starts", "prefill"])
def test_places_count_after_an_eviction(pkv, kind, dtype):
    hq, hkv, n, budget, scale = 8, 2, 700, 300, D ** -0.5
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = (torch.randn((m, h, D), generator=g, device="cuda").to(dtype) for m, h in ((3, hq), (n, hkv), (n, hkv)))
    kc, vc = (torch.zeros((5, BS, hkv, D), dtype=dtype, device="cuda") for _ in range(2))
    weights = pkv.attention_weights(5, hkv)
    for b, block in enumerate((3, 0, 4)):
        live = min(BS, n - b * BS)
        kc[block, :live], vc[block, :live] = k[b * BS:b * BS + live], v[b * BS:b * BS + live]
    weights.copy_(torch.rand(weights.shape, generator=g, device="cuda"))
    table, length = torch.tensor([[3, 0, 4]], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    kept, now = pkv.pkv_evict_kvcache(kc, vc, weights, table, length, n, budget, first=4, recent=20)
    held = [torch.stack([x[kept[0, h].long(), h] for h in range(hkv)], 1) for x in (k, v)]
    assert not torch.equal(kept[0, 0], kept[0, 1])              # the heads have kept different tokens
    mods, asked = {}, {}
    if kind == "cap":
        mods = asked = dict(softcap=20.0)
    elif kind == "window":
        mods = asked = dict(window=100)
    elif kind == "slopes":
        mods = asked = dict(slopes=torch.linspace(0.001, 0.1, hq, device="cuda"))
    elif kind == "starts":
        starts = torch.tensor([150], dtype=torch.int32, device="cuda")
        mods, asked = dict(starts=starts), dict(key_starts=starts)
    eps = torch.finfo(dtype).eps / 2
    if kind == "prefill":                                       # the last three rows, at places 297 to 299
        call = pkv.pkv_prefill_varlen_mod_f16 if dtype == torch.float16 else pkv.pkv_prefill_varlen_mod
        cu = [torch.tensor([0, m], dtype=torch.int32, device="cuda") for m in (3, budget)]
        out = call(q, *cu, 3, budget, scale, k_cache=kc, v_cache=vc, block_tables=table, window=100)
        ref, p, bound, _ = R.attention_rows(q, *held, budget - 3, scale, window=100)
        size = torch.einsum("hnt,thd->nhd", p, held[1].double().abs().repeat_interleave(hq // hkv, 1))
        room = 2 * eps * ref.abs() + size * (eps + 2.0 ** -18) + bound + 2.0 ** -25   # p rounded to 16 bits
    else:
        call = pkv.pkv_decode_mod_f16 if dtype == torch.float16 else pkv.pkv_decode_mod
        out = call(q[:1], kc, vc, table, now, n, scale, pkv.decode_mod_workspace(1, n, hq, hkv), **asked)
        ref, _, bound, _ = R.attention_rows(q[:1], *held, budget - 1, scale, **mods)
        room = eps * ref.abs() + bound + 2.0 ** -25
    assert bool(((out.double() - ref).abs() <= room).all())
    assert pkv.pkv_device_error() == 0


def test_lengths_side_by_side_and_overlapping(pkv):
    hkv, n = 2, 400
    kc, vc = (torch.randn((6, BS, hkv, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    weights = pkv.attention_weights(6, hkv)
    tables = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n, n - 1, 7, 0, 0, 0], dtype=torch.int32, device="cuda")
    before = kc.clone()
    for at in (0, 1, 2):
        with pytest.raises(ValueError):
            pkv.pkv_evict_kvcache(kc, vc, weights, tables, lens[:3], n, 100, new_context_lens=lens[at:at + 3])
    with pytest.raises(ValueError):
        pkv.pkv_evict_kvcache(kc, vc, weights, tables, lens[2:5], n, 100, new_context_lens=lens[:3])
    assert torch.equal(kc, before) and lens.tolist() == [n, n - 1, 7, 0, 0, 0]
    pkv.pkv_evict_kvcache(kc, vc, weights, tables, lens[:3], n, 100, new_context_lens=lens[3:])
    assert lens.tolist() == [n, n - 1, 7, 100, 100, 7] and pkv.pkv_device_error() == 0
