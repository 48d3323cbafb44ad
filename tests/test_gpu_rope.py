"""Rotary positions on the GPU against the 64-bit definition: layouts, partial heads, far positions, strides, in place,
fused with the store."""
import pytest
import torch

import mods_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


def _names(pkv, dtype):
    f16 = dtype == torch.float16
    return (pkv.pkv_rope_f16 if f16 else pkv.pkv_rope,
            pkv.pkv_rope_store_kvcache_f16 if f16 else pkv.pkv_rope_store_kvcache)


def _rows(n, heads, dims, dtype, seed, pad=0, offset=0):
    """Rows of a wider buffer, so that they are strided and may be unaligned."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.randn((n, heads * dims + pad + offset), generator=g).to(dtype).cuda()
    return buf[:, offset:offset + heads * dims].unflatten(1, (heads, dims))


def _check(got, x, positions, freqs, interleaved, magnitude):
    ref = R.rope(x, positions.cpu(), freqs.cpu(), interleaved, magnitude)
    off = (got.detach().cpu().double() - ref).abs()
    bound = R.rope_bound(x, ref, freqs.numel(), interleaved, magnitude)
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hkv,dims,rot,pad,offset", [
    (1, 16, 8, 128, 128, 0, 0),
    (7, 16, 8, 128, 128, 2056, 0),
    (5, 32, 8, 128, 64, 8, 8),
    (9, 3, 1, 128, 96, 0, 0),       # six of eight pieces turned
    (6, 5, 2, 96, 32, 16, 0),       # six pieces to a head: some threads of a block idle
    (4, 2, 2, 64, 6, 0, 0),         # 3 pairs
    (3, 4, 1, 20, 20, 0, 0),
    (3, 2, 1, 128, 128, 1, 0),      # odd row stride
    (3, 2, 1, 128, 128, 0, 1),      # rows 2 bytes off
    (2, 1, 1, 1024, 1024, 0, 0),
    (2, 3, 0, 256, 256, 0, 0),      # queries alone
    (2500, 2, 1, 128, 128, 0, 0),   # four tokens to a block, the last block with fewer
    (2433, 2, 1, 64, 64, 4, 0),
])
def test_rope(pkv, dtype, interleaved, n, hq, hkv, dims, rot, pad, offset):
    rope, _ = _names(pkv, dtype)
    q = _rows(n, hq, dims, dtype, 1, pad, offset)
    k = _rows(n, hkv, dims, dtype, 2, pad, offset) if hkv else None
    g = torch.Generator().manual_seed(n)
    positions = torch.randint(0, 1 << 20, (n,), generator=g).cuda()
    freqs, _ = pkv.rope_frequencies(rot)
    qo, ko = rope(q, k, positions, freqs, interleaved=interleaved, magnitude=1.25)
    assert qo.is_contiguous() and qo.shape == q.shape and qo.dtype == dtype
    _check(qo, q, positions, freqs, interleaved, 1.25)
    assert torch.equal(qo[..., rot:], q[..., rot:])
    if hkv:
        _check(ko, k, positions, freqs, interleaved, 1.25)
    else:
        assert ko is None
    # in place, in the strided rows: the same bits
    q0, k0 = q.clone(), None if k is None else k.clone()
    around = q.storage_offset()
    a, b = rope(q, k, positions, freqs, interleaved=interleaved, magnitude=1.25, q_out=q, k_out=k)
    assert a is q and torch.equal(q, qo) and q.storage_offset() == around and not torch.equal(q, q0)
    assert k is None or (b is k and torch.equal(k, ko))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hkv,dims,rot", [(5, 4, 2, 128, 6), (1300, 3, 1, 128, 120), (3, 5, 2, 72, 72), (7, 3, 3, 40, 24),
                                               (4, 2, 1, 96, 90), (2, 40, 8, 1000, 998), (6, 1, 1, 8, 2), (2, 3, 1, 24, 16),
                                               (5000, 1, 1, 1024, 1022)])
def test_any_turned_part_and_in_place(pkv, dtype, interleaved, n, hq, hkv, dims, rot):
    """16-byte pieces that hold turned elements and copied ones, partners in other pieces; in place and to the cache."""
    rope, rope_store = _names(pkv, dtype)
    q, k, v = (_rows(n, h, dims, dtype, s, 8) for s, h in ((1, hq), (2, hkv), (3, hkv)))
    positions = torch.randint(0, 1 << 17, (n,), generator=torch.Generator().manual_seed(5)).cuda()
    freqs, _ = pkv.rope_frequencies(rot)
    qo, ko = rope(q, k, positions, freqs, magnitude=1.25, interleaved=interleaved)
    few = min(n, 9)
    _check(qo[:few], q[:few], positions[:few], freqs, interleaved, 1.25)
    _check(ko[:few], k[:few], positions[:few], freqs, interleaved, 1.25)
    # the same rows a pair at a time: 2 bytes off
    q1, k1 = (torch.empty((n, h * dims + 9), dtype=dtype, device="cuda")[:, 1:1 + h * dims].unflatten(1, (h, dims))
              for h in (hq, hkv))
    q1.copy_(q)
    k1.copy_(k)
    qs, ks = rope(q1, k1, positions, freqs, magnitude=1.25, interleaved=interleaved)
    assert torch.equal(qo, qs) and torch.equal(ko, ks)
    slots = torch.randperm(n + 5, generator=torch.Generator().manual_seed(6))[:n].int().cuda()
    slots[n // 2] = -1
    kc, vc = (torch.full((n + 5, hkv, dims), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    q2 = rope_store(q, k, v, positions, freqs, kc, vc, slots, magnitude=1.25, interleaved=interleaved)
    kept = slots >= 0
    assert torch.equal(q2, qo)
    assert torch.equal(kc[slots[kept].long()], ko[kept]) and torch.equal(vc[slots[kept].long()], v[kept])
    assert int((kc == 3).all(-1).all(-1).sum()) == 5 + 1
    back = rope(q, k, positions, freqs, magnitude=1.25, interleaved=interleaved, q_out=q, k_out=k)
    assert back[0] is q and torch.equal(q, qo) and torch.equal(k, ko)
    assert pkv.pkv_device_error() == 0


def test_padding_between_rows_is_left(pkv):
    buf = torch.full((6, 2 * 128 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    q = buf[:, 8:264].unflatten(1, (2, 128))
    freqs, _ = pkv.rope_frequencies(128)
    pkv.pkv_rope(q, None, torch.arange(6, device="cuda"), freqs, q_out=q)
    assert bool((buf[:, :8] == 7).all()) and bool((buf[:, 264:] == 7).all())


@pytest.mark.parametrize("positions", [[0, 1, -1, -5000], [2 ** 24 + 1, 2 ** 31 + 7, 2 ** 40 + 3, 2 ** 62 - 1]])
def test_far_and_negative_positions(pkv, positions):
    q = _rows(4, 2, 128, torch.float16, 3)
    pos = torch.tensor(positions, device="cuda")
    freqs, _ = pkv.rope_frequencies(128)
    qo, _ = pkv.pkv_rope_f16(q, None, pos, freqs)
    _check(qo, q, pos, freqs, False, 1.0)


def test_special_values_stay_in_their_pair(pkv):
    q = _rows(3, 1, 128, torch.bfloat16, 4)
    q[1, 0, 5] = float("nan")
    q[2, 0, 70] = float("inf")
    freqs, _ = pkv.rope_frequencies(128)
    qo, _ = pkv.pkv_rope(q, None, torch.tensor([1, 2, 3], device="cuda"), freqs)
    bad = ~torch.isfinite(qo)
    want = torch.zeros_like(bad)
    want[1, 0, 5] = want[1, 0, 69] = want[2, 0, 6] = want[2, 0, 70] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hkv,dims,rot,pad", [(37, 16, 8, 128, 128, 2056), (3, 12, 12, 128, 64, 0),
                                                  (2600, 4, 1, 128, 128, 0), (5, 2, 1, 80, 10, 3), (4, 0, 2, 128, 128, 0)])
def test_rope_store_is_rope_then_store(pkv, dtype, interleaved, n, hq, hkv, dims, rot, pad):
    rope, rope_store = _names(pkv, dtype)
    q, k, v = (_rows(n, h, dims, dtype, s, pad) for s, h in ((1, hq), (2, hkv), (3, hkv)))
    g = torch.Generator().manual_seed(5)
    positions = torch.randint(0, 1 << 17, (n,), generator=g).cuda()
    freqs, _ = pkv.rope_frequencies(rot)
    blocks = n // 256 + 2
    slots = torch.randperm(blocks * 256, generator=g)[:n].int()
    slots[n // 2] = -1
    slots = slots.cuda()
    caches = [torch.full((blocks, 256, hkv, dims), 3.0, dtype=dtype, device="cuda") for _ in range(4)]
    qo, ko = rope(q, k, positions, freqs, interleaved=interleaved)
    pkv.pkv_store_kvcache(ko, v.contiguous(), caches[0], caches[1], slots)
    k_before = k.clone()
    q2 = rope_store(q, k, v, positions, freqs, caches[2], caches[3], slots, interleaved=interleaved)
    assert torch.equal(q2, qo) and torch.equal(k, k_before)
    assert torch.equal(caches[2], caches[0]) and torch.equal(caches[3], caches[1])
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [1300, 2500, 4999, 9000])
def test_many_tokens_are_as_few(pkv, dtype, interleaved, n):
    """Two, four and eight tokens to a block, the last one with fewer, against calls with one token to a block."""
    rope, rope_store = _names(pkv, dtype)
    q, k, v = (_rows(n, h, 128, dtype, s, 40) for s, h in ((1, 5), (2, 3), (3, 3)))
    positions = torch.randint(-9, 1 << 20, (n,), generator=torch.Generator().manual_seed(5)).cuda()
    freqs, _ = pkv.rope_frequencies(96)
    slots = torch.randperm(n + 300, generator=torch.Generator().manual_seed(6))[:n].int().cuda()
    slots[3] = -1
    caches = [torch.full((n + 300, 3, 128), 3.0, dtype=dtype, device="cuda") for _ in range(4)]
    qo, ko = rope(q, k, positions, freqs, interleaved=interleaved)
    q2 = rope_store(q, k, v, positions, freqs, *caches[:2], slots, interleaved=interleaved)
    for a in range(0, n, 700):
        cut = slice(a, min(n, a + 700))
        qw, kw = rope(q[cut], k[cut], positions[cut], freqs, interleaved=interleaved)
        assert torch.equal(qo[cut], qw) and torch.equal(ko[cut], kw) and torch.equal(q2[cut], qw)
        rope_store(q[cut], k[cut], v[cut], positions[cut], freqs, *caches[2:], slots[cut], interleaved=interleaved)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    kept = slots >= 0
    assert torch.equal(caches[0][slots[kept].long()], ko[kept]) and torch.equal(caches[1][slots[kept].long()], v[kept])


def test_bad_slots_are_reported_and_skipped(pkv):
    q, k = _rows(3, 2, 128, torch.bfloat16, 1), _rows(3, 1, 128, torch.bfloat16, 2)
    kc = torch.zeros((1, 256, 1, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    freqs, _ = pkv.rope_frequencies(128)
    slots = torch.tensor([256, 4, -2], dtype=torch.int32, device="cuda")
    pos = torch.arange(3, device="cuda")
    qo = pkv.pkv_rope_store_kvcache(q, k, k, pos, freqs, kc, vc, slots)
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SLOT
    assert torch.equal(vc[0, 4], k[1]) and int((vc != 0).any(-1).sum()) == 1
    _check(qo, q, pos, freqs, False, 1.0)


def test_stream_and_graph(pkv):
    q, k, v = (_rows(33, h, 128, torch.bfloat16, s) for s, h in ((1, 4), (2, 2), (3, 2)))
    freqs, _ = pkv.rope_frequencies(128)
    pos = torch.arange(33, device="cuda")
    slots = torch.arange(33, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((1, 256, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a, _ = pkv.pkv_rope(q, k, pos, freqs, stream=side)
    side.synchronize()
    qo = torch.empty_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.pkv_rope_store_kvcache(q, k, v, pos, freqs, kc, vc, slots, q_out=qo)
    assert not bool(kc.any())
    pos.add_(100)                           # a replay reads what the inputs hold then
    graph.replay()
    torch.cuda.synchronize()
    _check(qo, q, pos, freqs, False, 1.0)
    _check(kc[0, :33], k, pos, freqs, False, 1.0)


def test_binding_refusals(pkv):
    q, k = _rows(3, 2, 128, torch.bfloat16, 1), _rows(3, 1, 128, torch.bfloat16, 2)
    freqs, _ = pkv.rope_frequencies(128)
    pos, slots = torch.arange(3, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    kc = torch.zeros((1, 256, 1, 128), dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: pkv.pkv_rope(q.cpu(), k, pos, freqs), lambda: pkv.pkv_rope(q.half(), k, pos, freqs),
        lambda: pkv.pkv_rope(q, k[:2], pos, freqs), lambda: pkv.pkv_rope(q, k, pos[:2], freqs),
        lambda: pkv.pkv_rope(q, k, pos.int(), freqs), lambda: pkv.pkv_rope(q, k, pos, freqs.double()),
        lambda: pkv.pkv_rope(q.transpose(1, 2), k, pos, freqs), lambda: pkv.pkv_rope(q, None, pos, freqs, k_out=k),
        lambda: pkv.pkv_rope(q, k, pos, freqs, q_out=k), lambda: pkv.pkv_rope(q[0], k, pos, freqs),
        lambda: pkv.pkv_rope_store_kvcache(q, k, k, pos, freqs, kc, kc[:, :, :, :64], slots),
        lambda: pkv.pkv_rope_store_kvcache(q, k, k, pos, freqs, kc.half(), kc.half(), slots),
        lambda: pkv.pkv_rope_store_kvcache(q, k, k, pos, freqs, kc, kc, slots.long()),
        lambda: pkv.pkv_rope_store_kvcache(q, k, k, pos, freqs, kc, kc, slots[:2]),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_rope(q, k, pos, pkv.rope_frequencies(256)[0])   # more than the head has
    assert e.value.status == -2
    empty = q[:0]
    a, b = pkv.pkv_rope(empty, k[:0], pos[:0], freqs)
    assert a.shape == (0, 2, 128) and b.shape == (0, 1, 128)
