"""Prefill with capped and biased scores, windows, documents and prefixes, any head counts, contiguous and paged keys,
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


class Case:
    """Sequences given as (cached tokens, new tokens); keys contiguous, or in a cache whose other slots are NaN."""

    def __init__(self, seqs, hq, hkv, dtype, seed=1, paged=True, sharp=2.0, spare=3):
        g = torch.Generator().manual_seed(seed)
        dev = torch.Generator(device="cuda").manual_seed(seed)
        self.seqs, self.hq, self.hkv, self.dtype, self.paged = seqs, hq, hkv, dtype, paged
        lk, lq = [c + n for c, n in seqs], [n for _, n in seqs]
        self.cu_q = [0] + torch.tensor(lq).cumsum(0).tolist()
        self.cu_k = [0] + torch.tensor(lk).cumsum(0).tolist()
        self.max_q, self.max_k = max(lq) + 3, max(lk) + 1
        rows = self.cu_q[-1] + spare           # rows behind the last sequence
        buf = (torch.randn((rows, (hq + 1) * D), generator=dev, device="cuda") * sharp).to(dtype)
        self.q = buf[:, :hq * D].unflatten(1, (hq, D))
        self.k, self.v = (torch.randn((max(1, self.cu_k[-1]), (hkv + 1) * D), generator=dev, device="cuda").to(dtype)
                          [:, :hkv * D].unflatten(1, (hkv, D)) for _ in range(2))
        if paged:
            blocks = sum(-(-n // BS) for n in lk) + 2
            order = torch.randperm(blocks, generator=g).tolist()
            width = max(1, max(-(-n // BS) for n in lk)) + 1
            self.tables = torch.full((len(seqs), width), 99999999, dtype=torch.int32)
            self.kc, self.vc = (torch.full((blocks, BS, hkv, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
            at = 0
            for b, n in enumerate(lk):
                for j in range(-(-n // BS)):
                    self.tables[b, j] = order[at]
                    live = min(BS, n - j * BS)
                    first = self.cu_k[b] + j * BS
                    self.kc[order[at], :live], self.vc[order[at], :live] = (x[first:first + live] for x in (self.k, self.v))
                    at += 1

    def set_v(self, b, t, head, dim, value):
        self.v[self.cu_k[b] + t, head, dim] = value
        if self.paged:
            self.vc[int(self.tables[b, t // BS]), t % BS, head, dim] = value

    def run(self, pkv, scale=D ** -0.5, out=None, stream=None, **mods):
        fn = pkv.pkv_prefill_varlen_mod_f16 if self.dtype == torch.float16 else pkv.pkv_prefill_varlen_mod
        keys = (dict(k_cache=self.kc, v_cache=self.vc, block_tables=self.tables.cuda()) if self.paged
                else dict(k=self.k, v=self.v))
        cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (self.cu_q, self.cu_k)]
        return fn(self.q, *cu, self.max_q, self.max_k, scale, out=out, stream=stream, **keys, **mods)

    def check(self, out, scale=D ** -0.5, prefix_lens=None, key_starts=None, **mods):
        """p is rounded to 16 bits for the product with V: q = p (1 + e) with |e| at most half a step, eps. The result is
        sum q v / sum p or, where few keys are seen, sum q v / sum q. The first is off by sum p e v, at most eps sum p |v|;
        the second by sum p e (v - result), at most eps (sum p |v| + |result|). The polynomials for tanh are off by 6.9e-6
        (bf16) or 6.1e-7 (fp16) of a score, which the cap bounds; then the result's own rounding, eps |result|."""
        worst = 0.0
        eps = torch.finfo(self.dtype).eps / 2
        for b, (c, n) in enumerate(self.seqs):
            if n == 0:
                continue
            q0, k0, total = self.cu_q[b], self.cu_k[b], c + n
            for a in range(0, n, 2048):
                z = min(n, a + 2048)
                starts = None if key_starts is None else key_starts[q0 + a:q0 + z]
                ref, p, bound, off = R.attention_rows(
                    self.q[q0 + a:q0 + z], self.k[k0:k0 + total], self.v[k0:k0 + total], c + a, scale, starts=starts,
                    prefix=0 if prefix_lens is None else int(prefix_lens[b]), **mods)
                cap = (6.9e-6 if self.dtype == torch.bfloat16 else 6.1e-7) * mods.get("softcap", 0.0)
                size = torch.einsum("hnt,thd->nhd", p, self.v[k0:k0 + total].double().abs().nan_to_num(0, 0, 0)
                                    .repeat_interleave(self.hq // self.hkv, 1))
                room = ref.abs() * 2 * eps + size * (eps + 2 * cap + 2.0 ** -18) + bound + 2.0 ** -25
                got = out[q0 + a:q0 + z].double()
                err = (got - ref).abs()
                assert bool((err <= room).all()), (b, a, float((err / room).max()))
                # on the whole, what independent roundings leave
                norm = float(ref.norm())
                if norm > 0:
                    worst = max(worst, float(err.norm()) / norm)
        assert worst <= 2 * eps, worst


SEQS = {
    "one": [(0, 1)], "short": [(0, 1), (0, 2), (0, 127), (0, 128), (0, 129), (0, 0), (0, 255), (0, 256), (0, 257)],
    "cached": [(1, 1), (255, 1), (256, 300), (300, 0), (513, 130), (1000, 5)], "long": [(700, 1500)],
    "many": [((13 * i) % 90, (7 * i) % 41) for i in range(70)],
}
MODS = {
    "plain": {}, "cap": dict(softcap=5.0), "cap50": dict(softcap=50.0), "slopes": dict(slopes=True), "window": dict(window=100),
    "window1": dict(window=1), "docs": dict(key_starts=True), "prefix": dict(prefix_lens=True),
    "all": dict(softcap=30.0, slopes=True, window=333, key_starts=True, prefix_lens=True),
}


def _mods(mods, case, seed=3):
    g = torch.Generator().manual_seed(seed)
    mods = dict(mods)
    if mods.get("slopes"):
        mods["slopes"] = (torch.rand(case.hq, generator=g) * 0.2).cuda()
    if mods.get("prefix_lens"):
        mods["prefix_lens"] = torch.tensor([(0, 60, 150, 10 ** 6, -1)[b % 5] for b in range(len(case.seqs))],
                                           dtype=torch.int32, device="cuda")
    if mods.get("key_starts"):
        starts = []
        for c, n in case.seqs:           # documents of 1..250 tokens; some rows see nothing (a start behind them)
            at, doc = 0, []
            while at < c + n:
                size = int(torch.randint(1, 250, (1,), generator=g))
                doc += [at] * size
                at += size
            doc = doc[c:c + n]
            if n > 3:
                doc[2] = 10 ** 9
                doc[n // 2] = c + n // 2 + 1
                doc[0] = -5
            starts += doc
        mods["key_starts"] = torch.tensor(starts + [0] * (case.q.shape[0] - len(starts)), dtype=torch.int32, device="cuda")
    return mods


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("mods", list(MODS))
@pytest.mark.parametrize("seqs", list(SEQS))
def test_lengths_and_mods(pkv, seqs, mods, paged):
    dtype = torch.float16 if (len(mods) + len(seqs)) % 2 else torch.bfloat16
    c = Case(SEQS[seqs], 16, 8, dtype, seed=len(seqs), paged=paged)
    m = _mods(MODS[mods], c)
    out = torch.full((c.q.shape[0], 16, D), 7.0, dtype=dtype, device="cuda")
    assert c.run(pkv, out=out, **m) is out
    c.check(out, **m)
    assert bool((out[c.cu_q[-1]:] == 7).all())           # rows behind the last sequence are left
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (12, 12), (9, 3), (4, 1), (20, 2), (10, 2), (7, 1), (64, 8)])
def test_heads(pkv, hq, hkv, dtype):
    for paged in (False, True):
        c = Case([(0, 1), (40, 300), (300, 129), (0, 128), (7, 256), (0, 0)], hq, hkv, dtype, seed=hq, paged=paged)
        for mods in (MODS["all"], {}):
            m = _mods(mods, c)
            c.check(c.run(pkv, **m), **m)
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("sharp,scale,cap", [(2.0, D ** -0.5, 5.0), (4.0, D ** -0.5, 20.0), (60.0, 1.0, 50.0),
                                             (1.0, 1e-5, 30.0), (3.0, 1.0, 1e-3), (1.0, D ** -0.5, 1e6), (40.0, 1.0, 0.0)])
def test_cap_over_its_whole_range(pkv, sharp, scale, cap):
    for dtype in (torch.bfloat16, torch.float16):
        c = Case([(130, 200)], 4, 2, dtype, sharp=sharp)
        c.check(c.run(pkv, scale=scale, softcap=cap), scale=scale, softcap=cap)


@pytest.mark.parametrize("cap", [1e-40, 1e-20, 1e-9, 1e12, 1e31, 3e38])
def test_caps_of_any_size(pkv, cap):
    """Scores of 0 among them, which stay 0 under any cap."""
    for dtype in (torch.bfloat16, torch.float16):
        c = Case([(130, 200), (0, 140)], 4, 2, dtype)
        c.q[200:] = 0
        c.q[7] = 0
        c.check(c.run(pkv, softcap=cap), softcap=cap)


def test_matches_pkv_prefill(pkv):
    c = Case([(300, 400), (0, 77)], 16, 8, torch.bfloat16)
    cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (c.cu_q, c.cu_k)]
    n = c.cu_q[-1]
    a = pkv.pkv_prefill_varlen(c.q[:n], *cu, c.max_q, c.max_k, D ** -0.5, k_cache=c.kc, v_cache=c.vc, block_tables=c.tables.cuda())
    b = c.run(pkv)[:n]
    # Either rounds p (half a step, 2^-8 of each, so 2^-8 of sum p |v| <= 2^-8 max |v| in all) and its result (2^-8 of it).
    assert bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * (a.float().abs() + float(c.v.abs().max()))).all())


def test_matches_decode(pkv):
    """The last row of each sequence is what a decode over the same cache gives, up to p's rounding."""
    c = Case([(300, 40), (0, 77), (600, 1)], 8, 2, torch.float16)
    slopes = torch.linspace(0.01, 0.2, 8, device="cuda")
    out = c.run(pkv, softcap=20.0, slopes=slopes, window=250)
    last = torch.tensor([x - 1 for x in c.cu_q[1:]], device="cuda")
    ctx = torch.tensor([a + n for a, n in c.seqs], dtype=torch.int32, device="cuda")
    dec = pkv.pkv_decode_mod_f16(c.q[last], c.kc, c.vc, c.tables.cuda(), ctx, 1024, D ** -0.5,
                                 pkv.decode_mod_workspace(3, 1024, 8, 2), softcap=20.0, slopes=slopes, window=250)
    # p rounded to fp16 on one side (2^-11 of sum p |v|), both results rounded (2^-11 of them, at most max |v|)
    assert bool(((out[last].float() - dec.float()).abs() <= 3 * 2.0 ** -11 * float(c.v.abs().max())).all())


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (3, 1)])
def test_values_behind_the_mask(pkv, paged, hq, hkv):
    """NaN and infinities in V reach the rows that see their key, in their dim, and no others."""
    for mods in ({}, dict(window=50), dict(key_starts=True), dict(prefix_lens=True, softcap=9.0, slopes=True)):
        c = Case([(100, 300), (0, 200)], hq, hkv, torch.bfloat16, paged=paged)
        m = _mods(mods, c)
        clean = c.run(pkv, **m)
        spots = [(0, 250, 0, 9, float("nan")), (0, 399, hkv - 1, 70, float("inf")), (1, 64, 0, 127, float("-inf"))]
        for s in spots:
            c.set_v(*s)
        out = c.run(pkv, **m)
        bad = torch.zeros_like(out, dtype=torch.bool)
        for b, t, h, dim, _ in spots:
            cached, n = c.seqs[b]
            for i in range(n):
                p, r = cached + i, c.cu_q[b] + i
                sees = t <= p or ("prefix_lens" in m and t < int(m["prefix_lens"][b]))
                sees = sees and p - t < (m.get("window") or 10 ** 9)
                if "key_starts" in m:
                    sees = sees and t >= int(m["key_starts"][r])
                if sees:
                    bad[r, h * (hq // hkv):(h + 1) * (hq // hkv), dim] = True
        n = c.cu_q[-1]
        assert torch.equal(~torch.isfinite(out[:n]), bad[:n])
        # rows computed again do not round p: 2^-8 of sum p |v| apart, and one rounding of either result
        room = 2.0 ** -7 * (clean[:n].float().abs() + float(c.v.abs().nan_to_num(0, 0, 0).max()))
        assert bool(((out[:n].float() - clean[:n].float()).abs() <= room)[~bad[:n]].all())
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("mods", list(MODS))
@pytest.mark.parametrize("seqs", [[(0, 130), (300, 77), (0, 3)], [(2100, 140)]])
def test_what_lies_behind_a_sequence_changes_no_bit(pkv, seqs, mods):
    for dtype in (torch.bfloat16, torch.float16):
        for paged in (False, True):
            c = Case(seqs, 4, 2, dtype, paged=paged)
            m = _mods(MODS[mods], c)
            outs = []
            for value in (float("nan"), 0.0, 30000.0):
                if paged:
                    for b, (cached, new) in enumerate(seqs):
                        last = int(c.tables[b, (cached + new - 1) // BS])
                        for cache in (c.kc, c.vc):
                            cache[last, (cached + new - 1) % BS + 1:] = value
                outs.append(c.run(pkv, **m)[:c.cu_q[-1]])
            if not paged:  # the keys of the sequences behind the first one
                first = outs[0][:c.cu_q[1]].clone()
                for x in (c.k, c.v):
                    x[c.cu_k[1]:] *= 1000
                outs = [first, c.run(pkv, **m)[:c.cu_q[1]]]
            assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_nan_keys_and_queries(pkv):
    c = Case([(0, 200)], 4, 2, torch.float16, paged=False)
    c.k[150, 1, 3] = float("nan")
    c.q[20, 0, 5] = float("nan")
    out = c.run(pkv)[:200]
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[150:, 2:] = True
    bad[20, 0] = True
    assert torch.equal(torch.isnan(out), bad)


def test_bad_blocks_and_lengths(pkv):
    c = Case([(300, 40), (0, 77)], 4, 2, torch.bfloat16)
    good = c.run(pkv)
    tables = c.tables.clone()
    for bad in (-1, c.kc.shape[0], 2 ** 31 - 1):
        c.tables[0, 1] = bad
        out = c.run(pkv)
        assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_BLOCK
        assert torch.equal(out[40:117], good[40:117])
    c.tables = tables
    for field, value in (("cu_q", [0, 40, 39]), ("cu_q", [0, 500, 577]), ("cu_k", [0, 30, 107]), ("cu_q", [-1, 40, 117])):
        keep = getattr(c, field)
        setattr(c, field, value)
        c.run(pkv)
        assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN
        setattr(c, field, keep)
    c.max_q = 39
    c.run(pkv)
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN


def test_graph_and_streams(pkv):
    c = Case([(300, 400), (0, 77), (20, 130)], 8, 2, torch.bfloat16)
    m = _mods(MODS["all"], c)
    want = c.run(pkv, **m)
    out = torch.zeros_like(want)
    cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (c.cu_q, c.cu_k)]
    tables = c.tables.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.pkv_prefill_varlen_mod(c.q, *cu, c.max_q, c.max_k, D ** -0.5, k_cache=c.kc, v_cache=c.vc, block_tables=tables,
                                   out=out, **m)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:c.cu_q[-1]], want[:c.cu_q[-1]])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [c.run(pkv, stream=streams[i % 2], **m) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(o[:c.cu_q[-1]], want[:c.cu_q[-1]]) for o in outs)


def test_binding_refusals(pkv):
    c = Case([(3, 4)], 4, 2, torch.bfloat16)
    cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (c.cu_q, c.cu_k)]
    f = torch.zeros
    def call(q=c.q, cq=cu[0], ck=cu[1], scale=0.1, **kw):
        kw = kw or dict(k=c.k, v=c.v)
        if "k" not in kw and "block_tables" not in kw:
            kw.update(k=c.k, v=c.v)
        return pkv.pkv_prefill_varlen_mod(q, cq, ck, 8, 8, scale, **kw)
    call()
    tables = c.tables.cuda()
    bad = [dict(q=c.q.half()), dict(q=c.q.cpu()), dict(cq=cu[0].long()), dict(ck=cu[1][:1]), dict(k=None, v=None),
           dict(k=c.k[:2], v=c.v), dict(k=c.k, v=c.v.contiguous()), dict(block_tables=tables),
           dict(block_tables=tables, k_cache=c.kc, v_cache=c.vc, k=c.k, v=c.v), dict(slopes=f(3, device="cuda")), dict(slopes=f(4)),
           dict(block_tables=tables[0], k_cache=c.kc, v_cache=c.vc), dict(key_starts=f(2, dtype=torch.int32, device="cuda")),
           dict(prefix_lens=f(0, dtype=torch.int32, device="cuda")), dict(prefix_lens=f(1, device="cuda")), dict(out=c.q)]
    for kw in bad:
        with pytest.raises((ValueError, AttributeError)):
            call(**kw)
    for kw in (dict(softcap=-1.0), dict(softcap=float("inf")), dict(window=-1), dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(pkv.PkvError) as e:
            call(**kw)
        assert e.value.status == -6
    assert call(q=c.q[:0]).shape == (0, 4, 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("mods", list(MODS))
@pytest.mark.parametrize("seqs,hq,hkv", [
    ([(2500, 200)], 16, 8), ([(3000, 1)], 4, 1), ([(1000, 130), (0, 5), (2000, 64)], 3, 1), ([(900, 300), (0, 0)], 12, 12),
    ([(7, 2600)], 16, 8),           # full rounds of tiles and a rest
    ([(1500, 129), (20, 3)], 2, 1),
])
def test_split_keys(pkv, seqs, hq, hkv, dtype, mods):
    """Few query tiles, or few beyond whole rounds of them: their keys are split over clusters of CTAs."""
    c = Case(seqs, hq, hkv, dtype, seed=hq + len(seqs))
    m = _mods(MODS[mods], c)
    out = torch.full((c.q.shape[0], hq, D), 7.0, dtype=dtype, device="cuda")
    c.run(pkv, out=out, **m)
    c.check(out, **m)
    assert bool((out[c.cu_q[-1]:] == 7).all())
    assert torch.equal(c.run(pkv, **m)[:c.cu_q[-1]], out[:c.cu_q[-1]])
    assert pkv.pkv_device_error() == 0


def test_split_keys_values_behind_the_mask(pkv):
    c = Case([(2000, 100)], 4, 2, torch.bfloat16)
    clean = c.run(pkv)
    c.set_v(0, 2050, 0, 9, float("nan"))
    c.set_v(0, 60, 1, 100, float("inf"))
    out = c.run(pkv)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[50:100, :2, 9] = True
    bad[:100, 2:, 100] = True
    assert torch.equal(~torch.isfinite(out[:100]), bad[:100])
    room = 2.0 ** -7 * (clean[:100].float().abs() + 8)
    assert bool(((out[:100].float() - clean[:100].float()).abs() <= room)[~bad[:100]].all())


def test_split_keys_in_a_graph_and_bad_blocks(pkv):
    """The launch of split items runs beside the one before it: what follows on the stream sees all of both."""
    c = Case([(7, 2600)], 16, 8, torch.bfloat16)
    want = c.run(pkv, softcap=20.0)
    out, seen = torch.zeros_like(want), torch.zeros_like(want)
    cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (c.cu_q, c.cu_k)]
    tables = c.tables.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.zero_()
        pkv.pkv_prefill_varlen_mod(c.q, *cu, c.max_q, c.max_k, D ** -0.5, k_cache=c.kc, v_cache=c.vc, block_tables=tables,
                                   softcap=20.0, out=out)
        seen.copy_(out)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(seen[:2600], want[:2600])
    c.tables[0, 3] = -1
    c.run(pkv)
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_BLOCK
    c.tables[0, 3] = int(tables[0, 3])
    c.cu_q[1] = 2700          # more rows than q has
    c.run(pkv)
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN
