"""The 4-bit cache's store and load against the definition in 64 bits: the
stored bytes exactly, the values read back to half a step of their type."""
import numpy as np
import pytest
import torch

import q4_reference as R
import workloads as W

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


def calls(pkv, dtype):
    f16 = dtype == torch.float16
    return (pkv.pkv_store_kvcache_q4_f16 if f16 else pkv.pkv_store_kvcache_q4,
            pkv.pkv_load_kvcache_q4_f16 if f16 else pkv.pkv_load_kvcache_q4)


def poisoned(pkv, blocks, hkv):
    """Caches whose every byte is 0xff: codes 15, NaN scales and minima."""
    return tuple(pkv.q4_cache(blocks, hkv).fill_(0xff) for _ in range(2))


def check_bytes(cache, before, x, slots, is_v):
    """Every byte of the cache: the rows of the stored tokens, and the others as they were."""
    want = before.clone().cpu()
    code, s, z = (t.cpu() for t in R.quantise(x))
    for i, slot in enumerate(slots):
        if slot < 0:
            continue
        blk, tile, tok = slot // 256, slot % 256 // 16, slot % 16
        for h in range(x.shape[1]):
            at, b = R.row_bytes(code[i, h], s[i, h], z[i, h], tok, is_v)
            want[blk, h, tile, at] = b
    got = cache.cpu()
    nan = want.view(torch.int16).clone()
    # a NaN parameter may have any NaN's bits
    wp, gp = want[..., 1024:].contiguous().view(torch.float16), got[..., 1024:].contiguous().view(torch.float16)
    both = torch.isnan(wp) & torch.isnan(gp)
    zeros = (wp == 0) & (gp == 0)                      # either zero stands for 0
    assert torch.equal(want[..., :1024], got[..., :1024]), "codes"
    same = (wp.view(torch.int16) == gp.view(torch.int16)) | both | zeros
    assert bool(same.all()), "scales and minima"
    del nan


def check_rows(got, x, slots):
    """Rows read back: half a step of the type away from the 64-bit value, plus the fp32 rounding before it."""
    ref = R.dequantised(x)
    if got.dtype == torch.float16:
        ref = ref.clamp(-65504.0, 65504.0)
    half = torch.finfo(got.dtype).eps / 2
    live = torch.tensor([s >= 0 for s in slots], device=got.device)
    g, ref = got.double()[live], ref[live]
    assert torch.equal(torch.isnan(g), torch.isnan(ref))
    ok = (g - ref).abs() <= ref.abs() * (half + 2.0 ** -23) + 2.0 ** -25
    assert bool((ok | torch.isnan(ref)).all()), float((g - ref).abs().nan_to_num().max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,blocks,hkv,fused", [(1, 1, 8, True), (5, 2, 8, False), (33, 1, 1, True), (70, 3, 5, False),
                                                (300, 3, 2, True)])
def test_bytes_and_values(pkv, n, blocks, hkv, fused, dtype):
    dev = "cuda"
    gen = W.make_generator(n, dev)
    rng = np.random.default_rng(n)
    if fused:
        _, _, k, v = W.fused_qkv(n, gen, dev, hkv=hkv, dtype=dtype)
    else:
        k, v = W.normal((n, hkv, 128), gen, dev, dtype), W.normal((n, hkv, 128), gen, dev, dtype)
    slots = rng.permutation(blocks * 256)[:n].astype(np.int32)
    slots[rng.random(n) < 0.15] = -1
    store, load = calls(pkv, dtype)
    kc, vc = poisoned(pkv, blocks, hkv)
    kb, vb = kc.clone(), vc.clone()
    sm = torch.from_numpy(slots).to(dev)
    store(k, v, kc, vc, sm)
    check_bytes(kc, kb, k, slots, False)
    check_bytes(vc, vb, v, slots, True)
    # rows of slot -1 keep what they hold
    ko, vo = torch.full_like(k, 7.0, memory_format=torch.contiguous_format), torch.full((n, hkv, 128), 7.0, dtype=dtype, device=dev)
    load(kc, vc, sm, k=ko, v=vo)
    check_rows(ko, k, slots)
    check_rows(vo, v, slots)
    dead = torch.from_numpy(slots < 0).to(dev)
    assert bool((ko[dead] == 7).all()) and bool((vo[dead] == 7).all())
    assert pkv.pkv_device_error() == 0


def tie_rows(dtype, dev):
    """Rows full of elements on and next to the borders between codes: s is a power of two times small odd numbers and the
    elements are multiples of s / 4, with outliers of several sizes next to them."""
    rows = []
    rng = np.random.default_rng(1)
    for m in (1.0, 1.5, 1.25, 0.75, 3.0):
        for off in (0.0, -7.5, 3.0, -96.0):
            x = rng.integers(0, 61, 128) * m / 4 + off * m
            x[::32], x[1::32] = off * m, off * m + 15 * m      # the groups' min and max: s = m exactly
            rows.append(x)
    for big in (1.0, 300.0, 3e4):
        x = rng.standard_normal(128) * 1e-3
        x[::32] = big
        rows.append(x)
        rows.append(-x)
    return torch.tensor(np.array(rows), dtype=torch.float64, device=dev).to(dtype)[:, None]


@pytest.mark.parametrize("dtype", TYPES)
def test_borders_between_codes(pkv, dtype):
    x = tie_rows(dtype, "cuda")
    n = x.shape[0]
    slots = np.arange(n, dtype=np.int32) * 3
    store, load = calls(pkv, dtype)
    kc, vc = poisoned(pkv, 1, 1)
    kb, vb = kc.clone(), vc.clone()
    store(x, x, kc, vc, torch.from_numpy(slots).cuda())
    check_bytes(kc, kb, x, slots, False)
    check_bytes(vc, vb, x, slots, True)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_random_rows_exact(pkv, dtype):
    """Codes of 8.4 M elements of mixed sizes through values read back: equal to the 64-bit definition's."""
    dev = "cuda"
    gen = W.make_generator(11, dev)
    n, hkv = 8192, 4
    x = torch.randn((n, hkv, 128), generator=gen, device=dev)
    x = x * torch.exp2(torch.randint(-12, 6, (n, hkv, 1), generator=gen, device=dev).float())
    x = x + torch.randint(-3, 4, (n, 1, 128), generator=gen, device=dev)
    x = x.to(dtype)
    store, load = calls(pkv, dtype)
    kc, vc = poisoned(pkv, n // 256, hkv)
    slots = torch.randperm(n, generator=gen, device=dev).int()
    store(x, x.flip(0), kc, vc, slots)
    ko, vo = load(kc, vc, slots)
    check_rows(ko, x, [0] * n)
    check_rows(vo, x.flip(0), [0] * n)
    # one code off would be a whole step s away: far more than the rounding of the values
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_special_values(pkv, dtype):
    """Zeros, constants, tiny and huge rows; NaN and infinities stay in their group."""
    x = torch.zeros((9, 1, 128), dtype=dtype, device="cuda")
    x[1] = 3.25
    x[2] = -0.0
    x[3, 0, :64] = torch.finfo(dtype).max
    x[3, 0, 64:] = -torch.finfo(dtype).max
    x[4, 0, 5], x[4, 0, 40], x[4, 0, 70] = float("nan"), float("inf"), float("-inf")
    x[5] = torch.linspace(-1, 1, 128, device="cuda").to(dtype)
    x[6] = (torch.arange(128, device="cuda") * 2.0 ** -24).to(dtype)       # s is subnormal in fp16
    x[7, 0, ::2], x[7, 0, 1::2] = torch.finfo(dtype).max, -torch.finfo(dtype).max
    x[8, 0, 3] = torch.finfo(dtype).tiny
    slots = np.arange(9, dtype=np.int32) + 250
    store, load = calls(pkv, dtype)
    kc, vc = poisoned(pkv, 2, 1)
    kb, vb = kc.clone(), vc.clone()
    sm = torch.from_numpy(slots).cuda()
    store(x, x, kc, vc, sm)
    check_bytes(kc, kb, x, slots, False)
    check_bytes(vc, vb, x, slots, True)
    ko, vo = load(kc, vc, sm)
    check_rows(ko, x, slots)
    check_rows(vo, x, slots)
    nan = torch.isnan(ko[4, 0])
    assert bool(nan[:96].all()) and not bool(nan[96:].any())


@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_rows(pkv, dtype):
    """Row strides that are not a multiple of 8 elements, and rows that start at any element."""
    dev = "cuda"
    base = W.normal((50, 3 * 128 + 3), W.make_generator(3, dev), dev, dtype)
    k, v = base[:, 3:].unflatten(1, (3, 128)), base[:, :-3].unflatten(1, (3, 128))
    slots = np.arange(50, dtype=np.int32)[::-1].copy()
    store, _ = calls(pkv, dtype)
    kc, vc = poisoned(pkv, 1, 3)
    kb, vb = kc.clone(), vc.clone()
    store(k, v, kc, vc, torch.from_numpy(slots).to(dev))
    check_bytes(kc, kb, k, slots, False)
    check_bytes(vc, vb, v, slots, True)


def test_bad_slots_are_reported_and_skipped(pkv):
    dev = "cuda"
    gen = W.make_generator(4, dev)
    k, v = W.normal_bf16((4, 2, 128), gen, dev), W.normal_bf16((4, 2, 128), gen, dev)
    kc, vc = poisoned(pkv, 2, 2)
    kb = kc.clone()
    slots = torch.tensor([512, -2, 2 ** 31 - 1, -1], dtype=torch.int32, device=dev)
    pkv.pkv_store_kvcache_q4(k, v, kc, vc, slots)
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SLOT
    assert torch.equal(kc, kb) and torch.equal(vc, kb)
    ko, vo = pkv.pkv_load_kvcache_q4(kc, vc, slots)
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SLOT
    assert not bool(ko.any()) and not bool(vo.any())


def test_slots_past_32_bit_offsets(pkv):
    """A pool of over 2^32 bytes each for K and V: the last block's rows come back, repeated slots too."""
    dev = "cuda"
    blocks = 2 ** 32 // (8 * 20480) + 2
    gen = W.make_generator(5, dev)
    k, v = W.normal_bf16((40, 8, 128), gen, dev), W.normal_bf16((40, 8, 128), gen, dev)
    kc, vc = pkv.q4_cache(blocks), pkv.q4_cache(blocks)
    slots = np.arange(40, dtype=np.int32) + blocks * 256 - 40
    sm = torch.from_numpy(slots).to(dev)
    pkv.pkv_store_kvcache_q4(k, v, kc, vc, sm)
    ko, vo = pkv.pkv_load_kvcache_q4(kc, vc, torch.cat((sm, sm)))
    check_rows(ko[:40], k, slots)
    check_rows(vo[40:], v, slots)
    assert pkv.pkv_device_error() == 0


def test_more_tokens_than_one_grid_dimension(pkv):
    """Over 65535 * 16 tokens in one call (one kv head)."""
    dev = "cuda"
    n = 65535 * 16 + 4097
    blocks = -(-n // 256)
    gen = W.make_generator(6, dev)
    k, v = W.normal_bf16((n, 1, 128), gen, dev), W.normal_bf16((n, 1, 128), gen, dev)
    kc, vc = pkv.q4_cache(blocks, 1), pkv.q4_cache(blocks, 1)
    sm = torch.arange(n, dtype=torch.int32, device=dev)
    pkv.pkv_store_kvcache_q4(k, v, kc, vc, sm)
    ko, vo = pkv.pkv_load_kvcache_q4(kc, vc, sm)
    check_rows(ko, k, [0] * n)
    check_rows(vo, v, [0] * n)
