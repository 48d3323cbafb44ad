"""Decode with capped and biased scores, windows and first visible keys, any head counts, and attention added up,
against the 64-bit definition."""
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


def _case(lens, hq, hkv, dtype, seed=1, sharp=2.0, pad_q=0, shared=0):
    """Caches whose slots that no sequence holds are NaN, tables with garbage behind what is read, and q."""
    g = torch.Generator().manual_seed(seed)
    blocks = sum(-(-n // BS) for n in lens) + 3
    order = torch.randperm(blocks, generator=g).tolist()
    width = max(1, max(-(-n // BS) for n in lens)) + 1
    tables = torch.full((len(lens), width), 123456789, dtype=torch.int32)
    kc, vc = (torch.full((blocks, BS, hkv, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    dev = torch.Generator(device="cuda").manual_seed(seed)
    at = 0
    for b, n in enumerate(lens):
        for j in range(-(-n // BS)):
            tables[b, j] = order[at]
            live = min(BS, n - j * BS)
            for c in (kc, vc):
                c[order[at], :live] = torch.randn((live, hkv, D), generator=dev, device="cuda").to(dtype)
            at += 1
    buf = (torch.randn((len(lens), hq * D + pad_q), generator=dev, device="cuda") * sharp).to(dtype)
    q = buf[:, :hq * D].unflatten(1, (hq, D))
    return q, kc, vc, tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def _decode(pkv, dtype):
    return pkv.pkv_decode_mod_f16 if dtype == torch.float16 else pkv.pkv_decode_mod


def _compare(out, q, kc, vc, tables, lens, scale, dtype, weights=None, before=None, key_starts=None, **mods):
    hkv = kc.shape[2]
    if weights is not None:
        want_w, room = before.double(), torch.zeros_like(before, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n == 0:
            assert not bool(out[b].any())
            continue
        k, v = R.cache_rows(kc, tables[b].tolist(), n), R.cache_rows(vc, tables[b].tolist(), n)
        starts = None if key_starts is None else key_starts[b:b + 1]
        ref, p, bound, off = R.attention_rows(q[b:b + 1], k, v, n - 1, scale, starts=starts, **mods)
        err = (out[b:b + 1].double() - ref).abs()
        room_out = ref.abs() * (torch.finfo(dtype).eps / 2) + bound + 2.0 ** -25
        assert bool((err <= room_out).all()), (b, n, float((err / room_out).max()))
        if weights is not None:
            blocks = tables[b, :-(-n // BS)].long()
            w = want_w[blocks].transpose(0, 1).flatten(1)
            w[:, n - 1] = 0
            share = p[:, 0].unflatten(0, (hkv, -1))
            w[:, :n] += share.sum(1)
            want_w[blocks] = w.unflatten(1, (-1, BS)).transpose(0, 1)
            r = torch.zeros_like(w)
            r[:, :n] = (share * (2 * off[:, 0] + 2.0 ** -19).unflatten(0, (hkv, -1))[..., None]).sum(1)
            room[blocks] = r.unflatten(1, (-1, BS)).transpose(0, 1)
    if weights is not None:
        err = (weights.double() - want_w).abs()
        assert bool((err <= room + want_w.abs() * 2.0 ** -23).all())


LENS = {
    "one": [1], "edges": [15, 16, 17, 0, 31, 33, 255, 256, 257, 0, 511, 512, 513], "long": [5003, 3, 700],
    "single_long": [9001], "many": [(37 * i) % 301 for i in range(300)], "more": [1 + (i % 5) for i in range(700)],
    "none": [0, 0, 0],
}
MODS = {
    "plain": {}, "cap": dict(softcap=5.0), "slopes": dict(slopes=True), "window": dict(window=100),
    "window1": dict(window=1), "starts": dict(key_starts=True),
    "all": dict(softcap=30.0, slopes=True, window=333, key_starts=True),
}


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("mods", list(MODS))
@pytest.mark.parametrize("lens", list(LENS))
def test_lengths_and_mods(pkv, lens, mods, weights):
    dtype = torch.float16 if len(mods) % 2 else torch.bfloat16
    _run(pkv, LENS[lens], 16, 8, dtype, MODS[mods], weights)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (12, 12), (9, 3), (4, 1), (20, 2), (16, 1), (40, 2), (33, 1), (64, 8),
                                    (640, 640), (1300, 1300)])
def test_heads(pkv, hq, hkv, dtype):
    lens = [1, 40, 777, 256, 0, 1300] if hkv < 100 else [20, 0, 33]
    _run(pkv, lens, hq, hkv, dtype, MODS["all"], True)
    _run(pkv, lens, hq, hkv, dtype, {}, False)


def _run(pkv, lens, hq, hkv, dtype, mods, weights, sharp=2.0):
    q, kc, vc, tables, ctx = _case(lens, hq, hkv, dtype, seed=len(lens) + hq, sharp=sharp, pad_q=64)
    mods = dict(mods)
    g = torch.Generator().manual_seed(7)
    if mods.pop("slopes", None):
        mods["slopes"] = (torch.rand(hq, generator=g) * 0.2).cuda()
    starts = None
    if mods.pop("key_starts", None):
        # from the first key to beyond the last one (rows that see nothing)
        starts = torch.tensor([(n * i) // 7 + (3 if i % 8 == 7 else 0) for i, n in zip(range(len(lens)), lens)],
                              dtype=torch.int32)
        starts = torch.minimum(starts, torch.tensor([n + 2 for n in lens], dtype=torch.int32)).cuda()
        for b, n in enumerate(lens):   # tokens in front of the first visible one may hold anything
            for j in range(-(-min(n, int(starts[b])) // BS)):
                block, end = int(tables[b, j]), min(BS, min(n, int(starts[b])) - j * BS)
                kc[block, :end] = float("inf")
                vc[block, :end] = float("nan")
    most = max(max(lens), 1) + 5
    pool = torch.rand((kc.shape[0], hkv, BS), generator=g).cuda() if weights else None
    before = None if pool is None else pool.clone()
    ws = pkv.decode_mod_workspace(len(lens), most, hq, hkv, weights=weights)
    ws.fill_(0xff)                     # what is in it does not count
    scale = D ** -0.5
    dec = _decode(pkv, dtype)
    kw = dict(mods, key_starts=starts)
    out = dec(q, kc, vc, tables, ctx, most, scale, ws, weights=pool, **kw)
    _compare(out, q, kc, vc, tables, lens, scale, dtype, pool, before, **kw)
    ws.fill_(0x11)
    again = dec(q, kc, vc, tables, ctx, most, scale, ws, **kw)
    assert torch.equal(out, again)     # the same bits, with or without weights
    assert pkv.pkv_device_error() == 0


def test_matches_pkv_decode(pkv):
    lens = [37, 256, 300, 511, 4000]
    q, kc, vc, tables, ctx = _case(lens, 16, 8, torch.bfloat16)
    a = pkv.pkv_decode(q, kc, vc, tables, ctx, 4096, D ** -0.5, pkv.decode_workspace(5, 4096))
    b = pkv.pkv_decode_mod(q, kc, vc, tables, ctx, 4096, D ** -0.5, pkv.decode_mod_workspace(5, 4096))
    # both are within one rounding of the same value, up to fp32's error
    assert bool(((a.float() - b.float()).abs() <= a.float().abs() * 2.0 ** -7 + 1e-4).all())


def test_values_that_reach_the_result(pkv):
    """An infinite or NaN value at a visible key spoils its dims, a NaN key its rows' heads, and nothing else."""
    lens = [40, 40, 40]
    q, kc, vc, tables, ctx = _case(lens, 4, 2, torch.bfloat16)
    vc[int(tables[0, 0]), 3, 1, 9] = float("nan")
    kc[int(tables[1, 0]), 39, 0, 0] = float("nan")
    out = pkv.pkv_decode_mod(q, kc, vc, tables, ctx, 64, 0.1, pkv.decode_mod_workspace(3, 64, 4, 2))
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[0, 2:, 9] = True
    want[1, :2] = True
    assert torch.equal(bad, want)


def test_extreme_scores(pkv):
    """Scores far beyond the cap, and uncapped ones in the thousands: a softmax of the largest."""
    for cap in (0.0, 50.0):
        lens = [300, 64]
        q, kc, vc, tables, ctx = _case(lens, 4, 1, torch.float16, sharp=60.0)
        out = pkv.pkv_decode_mod_f16(q, kc, vc, tables, ctx, 512, 1.0, pkv.decode_mod_workspace(2, 512, 4, 1),
                                     softcap=cap)
        _compare(out, q, kc, vc, tables, lens, 1.0, torch.float16, softcap=cap)


@pytest.mark.parametrize("cap", [1e-40, 1e-20, 1e-9, 1e-3, 1e12, 1e31, 3e38])
def test_caps_of_any_size(pkv, cap):
    """Scores of 0 among them, which stay 0 under any cap."""
    lens = [300, 64, 40]
    for dtype in (torch.bfloat16, torch.float16):
        q, kc, vc, tables, ctx = _case(lens, 4, 2, dtype)
        q[1] = 0
        kc[tables[2, 0], :7] = 0
        out = _decode(pkv, dtype)(q, kc, vc, tables, ctx, 512, D ** -0.5, pkv.decode_mod_workspace(3, 512, 4, 2), softcap=cap)
        _compare(out, q, kc, vc, tables, lens, D ** -0.5, dtype, softcap=cap)


def test_bad_blocks_and_lengths_are_reported(pkv):
    lens = [300, 40]
    q, kc, vc, tables, ctx = _case(lens, 4, 2, torch.bfloat16)
    ws = pkv.decode_mod_workspace(2, 512, 4, 2, weights=True)
    pool = pkv.attention_weights(kc.shape[0], 2)
    good = pkv.pkv_decode_mod(q, kc, vc, tables, ctx, 512, 0.1, ws, weights=pool)
    for bad in (-1, kc.shape[0], 2 ** 31 - 1):
        t = tables.clone()
        t[0, 1] = bad
        out = pkv.pkv_decode_mod(q, kc, vc, t, ctx, 512, 0.1, ws, weights=pool)
        assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_BLOCK
        assert torch.equal(out[1], good[1])
    for n in (-1, 513, 2 ** 31 - 1):
        c = ctx.clone()
        c[0] = n
        out = pkv.pkv_decode_mod(q, kc, vc, tables, c, 512, 0.1, ws, weights=pool)
        assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN
        assert torch.equal(out[1], good[1]) and not bool(out[0].any())
    assert pkv.pkv_device_error() == 0


def test_graph_streams_and_new_lengths(pkv):
    """Captured once, replayed with other lengths; two captured calls with workspaces of their own on two streams."""
    lens = [300, 40, 0, 700]
    q, kc, vc, tables, ctx = _case(lens, 8, 2, torch.bfloat16)
    scale = D ** -0.5
    out, pool = torch.empty_like(q), pkv.attention_weights(kc.shape[0], 2)
    ws = pkv.decode_mod_workspace(4, 800, 8, 2, weights=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.pkv_decode_mod(q, kc, vc, tables, ctx, 800, scale, ws, softcap=20.0, weights=pool, out=out)
    for new in (lens, [17, 40, 0, 1], [0, 0, 0, 0], [299, 1, 0, 699]):
        ctx.copy_(torch.tensor(new, dtype=torch.int32))
        before = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        _compare(out, q, kc, vc, tables, new, scale, torch.bfloat16, pool, before, softcap=20.0)
    ctx.copy_(torch.tensor(lens, dtype=torch.int32))
    want = pkv.pkv_decode_mod(q, kc, vc, tables, ctx, 800, scale, ws)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [pkv.decode_mod_workspace(4, 800, 8, 2) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        outs.append(pkv.pkv_decode_mod(q, kc, vc, tables, ctx, 800, scale, spaces[i % 2], stream=streams[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert pkv.pkv_device_error() == 0


def test_weights_add_up_over_steps(pkv):
    """A sequence that grows by a token a step: the sums are those of all its steps, each token's from its own step on."""
    n0, steps = 250, 12
    q, kc, vc, tables, _ = _case([n0 + steps], 4, 2, torch.bfloat16)
    pool = torch.full((kc.shape[0], 2, BS), 5.0, device="cuda")
    ws = pkv.decode_mod_workspace(1, 300, 4, 2, weights=True)
    want = torch.full((2, n0 + steps), 5.0, dtype=torch.float64, device="cuda")
    for n in range(n0 + 1, n0 + steps + 1):
        ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
        pkv.pkv_decode_mod(q, kc, vc, tables, ctx, 300, 0.1, ws, weights=pool)
        k, v = R.cache_rows(kc, tables[0].tolist(), n), R.cache_rows(vc, tables[0].tolist(), n)
        _, p, _, _ = R.attention_rows(q, k, v, n - 1, 0.1)
        want[:, n - 1] = 0
        want[:, :n] += p[:, 0].unflatten(0, (2, -1)).sum(1)
    got = pool[tables[0, :2].long()].transpose(0, 1).flatten(1)[:, :n0 + steps].double()
    assert bool(((got - want).abs() <= want * 2.0 ** -16 + 2.0 ** -20).all())


def test_binding_refusals(pkv):
    q, kc, vc, tables, ctx = _case([5, 9], 4, 2, torch.bfloat16)
    ws = pkv.decode_mod_workspace(2, 64, 4, 2)
    f = torch.zeros
    def call(q=q, kc=kc, vc=vc, bt=tables, cl=ctx, ws=ws, **kw):
        return pkv.pkv_decode_mod(q, kc, vc, bt, cl, 64, 0.1, ws, **kw)
    call()
    bad = [dict(q=q.half()), dict(q=q.cpu()), dict(kc=kc[:, :, :, :64]), dict(vc=vc[:1]), dict(kc=kc.half()), dict(bt=tables.long()),
           dict(cl=ctx[:1]), dict(bt=tables[:1]), dict(ws=ws.float()), dict(slopes=f(3, device="cuda")), dict(slopes=f(4)),
           dict(slopes=f(4, device="cuda", dtype=torch.float64)), dict(key_starts=f(1, dtype=torch.int32, device="cuda")),
           dict(key_starts=f(2, device="cuda")), dict(weights=f((1, 2, 256), device="cuda")),
           dict(weights=f((kc.shape[0], 2, 256), device="cuda", dtype=torch.float16)), dict(out=torch.empty_like(q)[:, :2])]
    for kw in bad:
        with pytest.raises(ValueError):
            call(**kw)
    pool = pkv.attention_weights(kc.shape[0], 2)
    for kw, status in ((dict(softcap=-1.0), -6), (dict(window=-1), -6), (dict(softcap=float("nan")), -6),
                       (dict(ws=ws[:16]), -5), (dict(weights=pool), -5)):
        with pytest.raises(pkv.PkvError) as e:
            call(**kw)
        assert e.value.status == status
    assert call(q=q[:0]).shape == (0, 4, 128)
