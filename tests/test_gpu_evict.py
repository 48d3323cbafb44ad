"""Eviction from the paged cache: what stays, where it goes, what is left alone."""
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


def _weights(kind, shape, g):
    w = torch.rand(shape, generator=g)
    if kind == "ties":           # few values: most of them equal
        return torch.floor(w * 4)
    if kind == "zeros":
        return torch.zeros(shape) * torch.where(w < 0.5, -1.0, 1.0)   # of both signs
    if kind == "wide":           # all exponents, subnormals, negative ones, infinities and NaN
        x = torch.exp((w - 0.5) * 170) * torch.where(torch.rand(shape, generator=g) < 0.2, -1.0, 1.0)
        x[w < 0.02] = float("nan")
        x[(w > 0.5) & (w < 0.51)] = float("inf")
        x[(w > 0.6) & (w < 0.61)] = float("-inf")
        return x
    return w ** 8


def _case(lens, hkv, kind, seed, dtype=torch.bfloat16, new=0):
    g = torch.Generator().manual_seed(seed)
    old = sum(-(-n // BS) for n in lens) + 2
    blocks = old + new
    order = torch.randperm(old, generator=g).tolist()
    width = max(1, max(-(-n // BS) for n in lens))
    tables, at = torch.full((len(lens), width), -7, dtype=torch.int32), 0
    for b, n in enumerate(lens):
        k = -(-n // BS)
        tables[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
        at += k
    dev = torch.Generator(device="cuda").manual_seed(seed)
    kc, vc = (torch.randn((blocks, BS, hkv, D), generator=dev, device="cuda").to(dtype) for _ in range(2))
    w = _weights(kind, (blocks, hkv, BS), g).cuda()
    return kc, vc, w, tables, old, g


def _expect(kc, vc, w, tables, to, lens, first, recent, budget):
    """The caches, weights and kept positions after the call, one row at a time."""
    hkv = kc.shape[2]
    ek, ev, ew = kc.clone(), vc.clone(), w.clone()
    kept = torch.full((len(lens), hkv, budget), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        blocks = tables[b, :-(-n // BS)].long().cuda()
        flat_w = w[blocks].transpose(0, 1).flatten(1)[:, :n].cpu()
        for h in range(hkv):
            stay = R.evict_choice(flat_w[h].tolist(), first, recent, budget)
            kept[b, h, :len(stay)] = torch.tensor(stay, dtype=torch.int32)
            src = torch.tensor(stay, device="cuda")
            j = torch.arange(len(stay), device="cuda")
            fb, fi = blocks[src // BS], src % BS
            tb, ti = to[b].long().cuda()[j // BS], j % BS
            ek[tb, ti, h], ev[tb, ti, h], ew[tb, h, ti] = kc[fb, fi, h], vc[fb, fi, h], w[fb, h, fi]
    return ek, ev, ew, kept


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.int32 if a.dtype == torch.float32 else torch.int16),
                       b.contiguous().view(torch.int32 if b.dtype == torch.float32 else torch.int16))


CASES = [
    ([5], 1, 1, 0, 0), ([5], 1, 1, 1, 0), ([5], 1, 1, 0, 1), ([1, 2, 3, 0], 2, 2, 1, 1), ([300, 255, 256, 257, 0, 40], 2, 256, 4, 32),
    ([1000, 20, 700], 3, 100, 0, 0), ([1000, 999], 2, 1000, 10, 10), ([600], 5, 599, 0, 0), ([700, 800], 2, 300, 300, 0),
    ([700, 800], 2, 300, 0, 300), ([513] * 40, 8, 70, 3, 9), ([20001], 2, 5000, 4, 500), ([52000, 300], 1, 1025, 2, 3),
    ([900] * 30, 12, 450, 16, 64),
]


@pytest.mark.parametrize("kind", ["heavy", "ties", "zeros", "wide"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_evict(pkv, case, kind, in_place):
    lens, hkv, budget, first, recent = CASES[case]
    if kind == "wide" and max(lens) > 20000:
        pytest.skip("many values are covered by the shorter ones")
    need = [-(-min(n, budget) // BS) for n in lens]
    dtype = torch.float16 if case % 2 else torch.bfloat16
    kc, vc, w, tables, old, g = _case(lens, hkv, kind, case, dtype, 0 if in_place else sum(need) + 1)
    to = tables
    if not in_place:
        order = (old + torch.randperm(sum(need) + 1, generator=g)).tolist()
        to = torch.full((len(lens), max(1, -(-budget // BS))), -1, dtype=torch.int32)
        for b, k in enumerate(need):
            to[b, :k] = torch.tensor([order.pop() for _ in range(k)], dtype=torch.int32)
    want = _expect(kc, vc, w, tables, to, lens, first, recent, budget)
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kept, new_lens = pkv.pkv_evict_kvcache(kc, vc, w, tables.cuda(), ctx, max(lens), budget, first=first, recent=recent,
                                           new_block_tables=None if in_place else to.cuda())
    assert pkv.pkv_device_error() == 0
    assert new_lens.tolist() == [min(n, budget) for n in lens]
    assert torch.equal(kept.cpu(), want[3])
    assert _same(kc, want[0]) and _same(vc, want[1]) and _same(w, want[2])


def test_shared_blocks_to_new_ones(pkv):
    """Two sequences behind the same old blocks; each gets its own copy."""
    kc, vc, w, tables, old, _ = _case([600], 2, "heavy", 3, new=4)
    tables = tables.repeat(2, 1)
    to = torch.tensor([[old, old + 1], [old + 2, old + 3]], dtype=torch.int32)
    want = _expect(kc, vc, w, tables, to, [600, 520], 0, 8, 400)
    ctx = torch.tensor([600, 520], dtype=torch.int32, device="cuda")
    kept, _ = pkv.pkv_evict_kvcache(kc, vc, w, tables.cuda(), ctx, 700, 400, recent=8, new_block_tables=to.cuda())
    assert torch.equal(kept.cpu(), want[3]) and _same(kc, want[0]) and _same(vc, want[1]) and _same(w, want[2])


def test_bad_blocks_and_lengths(pkv):
    kc, vc, w, tables, old, _ = _case([600, 300], 2, "heavy", 4, new=4)
    to = torch.tensor([[old, old + 1], [old + 2, old + 3]], dtype=torch.int32)
    ctx = torch.tensor([600, 300], dtype=torch.int32, device="cuda")
    for bad in (-1, kc.shape[0], 2 ** 31 - 1):
        for which in (tables, to):
            t = which.clone()
            t[0, 1] = bad
            a, b = (t, to) if which is tables else (tables, t)
            kept, lens = pkv.pkv_evict_kvcache(kc, vc, w, a.cuda(), ctx, 700, 400, new_block_tables=b.cuda())
            assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_BLOCK
            assert lens.tolist() == [400, 300]
    for n in (-1, 701, 2 ** 31 - 1):
        c = torch.tensor([n, 300], dtype=torch.int32, device="cuda")
        kept, lens = pkv.pkv_evict_kvcache(kc, vc, w, tables.cuda(), c, 700, 400, new_block_tables=to.cuda())
        assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN
        assert lens.tolist() == [0, 300] and bool((kept[0] == -1).all())


def test_graph_and_stream(pkv):
    lens = [600, 300, 900]
    kc, vc, w, tables, old, _ = _case(lens, 2, "ties", 5, new=6)
    to = (old + torch.arange(6, dtype=torch.int32)).view(3, 2)
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kept = torch.empty((3, 2, 400), dtype=torch.int32, device="cuda")
    new_lens = torch.empty(3, dtype=torch.int32, device="cuda")
    td, nd = tables.cuda(), to.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.pkv_evict_kvcache(kc, vc, w, td, ctx, 900, 400, first=1, new_block_tables=nd, kept=kept,
                              new_context_lens=new_lens)
    w.copy_(_weights("heavy", tuple(w.shape), torch.Generator().manual_seed(9)))
    want = _expect(kc, vc, w, tables, to, lens, 1, 0, 400)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept.cpu(), want[3]) and _same(kc, want[0]) and _same(w, want[2])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other, _ = pkv.pkv_evict_kvcache(kc, vc, w, td, ctx, 900, 400, first=1, new_block_tables=nd, stream=side)
    side.synchronize()
    assert torch.equal(other, kept)


def test_binding_refusals(pkv):
    kc, vc, w, tables, old, _ = _case([600], 2, "heavy", 4, new=2)
    ctx, td = torch.tensor([600], dtype=torch.int32, device="cuda"), tables.cuda()
    nd = torch.tensor([[old, old + 1]], dtype=torch.int32, device="cuda")
    def call(kc=kc, vc=vc, w=w, t=td, c=ctx, budget=400, **kw):
        return pkv.pkv_evict_kvcache(kc, vc, w, t, c, 600, budget, **kw)
    bad = [dict(kc=kc.float()), dict(vc=vc[:1]), dict(w=w[:1]), dict(w=w.half()), dict(t=td.long()), dict(t=td[0]),
           dict(c=ctx.long()), dict(budget=0), dict(new_block_tables=nd[0]), dict(new_block_tables=nd.long()),
           dict(kept=torch.empty((1, 2, 399), dtype=torch.int32, device="cuda")), dict(new_context_lens=ctx),
           dict(new_context_lens=torch.empty(2, dtype=torch.int32, device="cuda"))]
    for kw in bad:
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(first=-1), dict(recent=-1), dict(first=401), dict(first=200, recent=201), dict(new_block_tables=nd[:, :1])):
        with pytest.raises(pkv.PkvError) as e:
            call(**kw)
        assert e.value.status == -6
    assert int(call(c=ctx[:0])[0].numel()) == 0
