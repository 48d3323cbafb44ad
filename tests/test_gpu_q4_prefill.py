"""Prefill over the 4-bit cache against attention in 64 bits over the values read
back, and beside loading the rows and running the 16-bit prefill."""
import numpy as np
import pytest
import torch

import q4_reference as R
import workloads as W
from test_gpu_q4_decode import Case

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


class Prefill(Case):
    """Sequences of lk tokens of which the last lq are queries."""

    def __init__(self, pkv, lq, lk, hq, hkv, dtype, seed=0, extra_rows=0, rows=None):
        super().__init__(pkv, lk, hq, hkv, dtype, seed, rows)
        gen = W.make_generator(seed + 1000, "cuda")
        self.lq, self.total = lq, sum(lq)
        self.cq = np.concatenate(([0], np.cumsum(lq))).astype(np.int32)
        self.ck = np.concatenate(([0], np.cumsum(lk))).astype(np.int32)
        qkv = W.normal((self.total + extra_rows, (hq + 2 * hkv) * 128), gen, "cuda", dtype)
        self.q = qkv[:, :hq * 128].unflatten(1, (hq, 128))
        self.d_cq, self.d_ck = torch.from_numpy(self.cq).cuda(), torch.from_numpy(self.ck).cuda()

    def prefill(self, **kw):
        return self.f("pkv_prefill_varlen_q4")(self.q, self.d_cq, self.d_ck, max(self.lq), max(self.lens), self.scale,
                                               self.kc, self.vc, self.tables, **kw)

    def check(self, out, only=None):
        assert self.pkv.pkv_device_error() == 0
        half = torch.finfo(self.dtype).eps / 2
        for b, n in enumerate(self.lens):
            if self.lq[b] == 0 or (only is not None and b not in only):
                continue
            a, e = self.first[b], self.first[b + 1]
            k, v = R.dequantised(self.k[a:e]).to(self.dtype), R.dequantised(self.v[a:e]).to(F16)
            q = self.q[self.cq[b]:self.cq[b + 1]]
            ref = R.attention(q, k, v, n - self.lq[b], self.scale)
            # k (of the rows' type) and v (fp16) as the products read them; p is rounded to fp16 (2^-11 of each weight),
            # the logits' fp32 sums are off by 2^-20 of their magnitude, the result is rounded once
            big = float(v.double().abs().amax())
            s = float((q.double().abs().amax((0, 1)) * k.double().abs().amax((0, 1))).sum()) * self.scale
            tol = half * ref.abs() + big * (2.0 ** -11 + 2.0 ** -20 * (2 + s))
            err = (out[self.cq[b]:self.cq[b + 1]].double() - ref).abs()
            assert bool((err <= tol).all()), f"sequence {b} ({self.lq[b]} of {n}): {float((err / tol).max()):.2f} of the bound"


SHAPES = [
    ([1], [1]), ([1], [129]), ([128], [128]), ([129, 1, 127], [129, 300, 383]), ([5, 200, 33], [5, 429, 256]),
    ([255, 257, 1, 64], [255, 513, 1024, 64]), ([0, 40, 0], [0, 40, 700]), ([700], [3000])]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lq,lk", SHAPES)
def test_against_64_bits(pkv, lq, lk, dtype):
    c = Prefill(pkv, lq, lk, 16, 8, dtype, seed=sum(lk)).fill()
    c.check(c.prefill())


@pytest.mark.parametrize("hq,hkv,dtype", [(2, 1, BF16), (32, 8, BF16), (12, 3, F16), (6, 3, F16)])
def test_head_layouts(pkv, hq, hkv, dtype):
    c = Prefill(pkv, [200, 130], [450, 130], hq, hkv, dtype, seed=hq).fill()
    c.check(c.prefill())


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_load_then_prefill(pkv, dtype):
    """As pkv_load_kvcache_q4 followed by the contiguous 16-bit prefill, which rounds v and p to the rows' type where
    this one takes fp16: at most 2^-8 (bf16) of the largest value each, and the results' own rounding."""
    c = Prefill(pkv, [300, 1, 129, 513], [1324, 700, 129, 2048], 16, 8, dtype, seed=21).fill()
    k, v = c.f("pkv_load_kvcache_q4")(c.kc, c.vc, c.slots)
    want = c.f("pkv_prefill_varlen")(c.q, c.d_cq, c.d_ck, max(c.lq), max(c.lens), c.scale, k=k, v=v)
    out = c.prefill()
    c.check(out)
    half = torch.finfo(dtype).eps / 2
    off = (out.double() - want.double()).abs()
    assert bool((off <= half * (2 * want.double().abs() + 2.5 * float(v.double().abs().max()))).all())
    plan = pkv.pkv_prefill_plan(c.cq, c.ck)
    assert torch.equal(c.prefill(plan=plan), out) and torch.equal(c.prefill(), out)


# Few query tiles behind many keys: the keys of a tile are split over 2, 4 or 8 CTAs.
SPLIT = [
    ([100], [6000]), ([1], [2500]), ([1, 100, 0], [1, 6000, 40]),      # parts without keys
    ([500, 3], [5000, 4990]),                                          # rows that see none of a part's keys
    ([300, 300, 40], [2348, 2300, 2048]),                              # 2 CTAs
    ([2560], [8560])]                                                  # whole rounds of tiles, then 8 split ones


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lq,lk", SPLIT)
def test_keys_split_over_ctas(pkv, lq, lk, dtype):
    c = Prefill(pkv, lq, lk, 16, 8, dtype, seed=31 + len(lq)).fill()
    out = c.prefill()
    c.check(out)
    assert torch.equal(c.prefill(), out)
    c.check(c.prefill(plan=pkv.pkv_prefill_plan(c.cq, c.ck)))


# 4 query tiles to a sequence on average and 28 key tiles: two CTAs widen each key tile for both.
@pytest.mark.parametrize("lq,lk,hq,hkv,dtype", [
    ([1100], [4000], 32, 8, BF16),                  # an odd number of tiles, the last of them not full
    ([2400, 200], [4600, 900], 32, 8, F16),         # pairs whose later tile, or both, have no row
    ([2100, 150], [2100, 4000], 32, 8, BF16),
    ([1152, 1025, 1030], [1300, 1025, 5000], 24, 12, F16)])
def test_pairs_of_query_tiles(pkv, lq, lk, hq, hkv, dtype):
    c = Prefill(pkv, lq, lk, hq, hkv, dtype, seed=50 + hq).fill()
    out = c.prefill()
    c.check(out)
    assert torch.equal(c.prefill(), out)
    planned = c.prefill(plan=pkv.pkv_prefill_plan(c.cq, c.ck))                  # (a plan's tiles are not paired)
    c.check(planned)
    if lq == [2100, 150]:                                                       # (elsewhere some tiles' keys are split)
        assert torch.equal(planned, out)


def test_pairs_nan_values_and_bad_blocks(pkv):
    c = Prefill(pkv, [2400, 300], [4500, 300], 32, 8, BF16, seed=56).fill()
    want = c.prefill()
    c.v[2100 + 2000, 1, 40] = float("nan")          # keys of either half of a tile: sequence 0, kv heads 1 and 2
    c.v[2100 + 2080, 2, 70] = float("nan")
    c.v[c.first[1] + 10, 0, 3] = float("inf")       # sequence 1, kv head 0
    out = c.fill().prefill()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[2000:2400, 4:8, 32:64] = True
    hit[2080:2400, 8:12, 64:96] = True
    hit[2410:2700, 0:4, 0:32] = True
    assert bool(out[hit].isnan().all())
    assert torch.equal(out[~hit], want[~hit])
    assert pkv.pkv_device_error() == 0
    c.tables[1, 0] = 10 ** 6
    out = c.prefill()
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_BLOCK
    assert torch.equal(out[:2400][~hit[:2400]], want[:2400][~hit[:2400]])


def test_split_heads_growing_logits_and_graph(pkv):
    """Other head layouts; maxima that differ from part to part; captured and replayed."""
    for hq, hkv in ((8, 1), (4, 2), (32, 8)):
        c = Prefill(pkv, [130, 7], [4400, 3000], hq, hkv, BF16, seed=40 + hq)
        c.k = (c.k.float() + torch.linspace(-3, 3, c.k.shape[0], device="cuda")[:, None, None]).to(BF16)
        c.q = c.q.abs()
        want = c.fill().prefill()
        c.check(want)
        out = torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.prefill(out=out)
        for _ in range(2):
            out.fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_split_nan_values_and_bad_blocks(pkv):
    lq, lk = [200, 50], [5000, 4000]
    c = Prefill(pkv, lq, lk, 4, 2, BF16, seed=45).fill()
    want = c.prefill()
    c.v[4900, 1, 40] = float("nan")                 # sequence 0, group 1 of kv head 1: rows at or past key 4900
    c.v[c.first[1] + 700, 0, 3] = float("inf")      # sequence 1, group 0 of kv head 0: every row
    out = c.fill().prefill()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[4900 - 4800:200, 2:4, 32:64] = True
    hit[200:250, 0:2, 0:32] = True
    assert bool(out[hit].isnan().all())
    assert torch.equal(out[~hit], want[~hit])
    assert pkv.pkv_device_error() == 0
    c.tables[1, 9] = 10 ** 6
    out = c.prefill()
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_BLOCK
    assert torch.equal(out[:200][~hit[:200]], want[:200][~hit[:200]])


def test_calls_at_once_and_captured(pkv):
    """Calls of all three kinds on several streams at once, and one captured graph of them."""
    cases = [Prefill(pkv, lq, lk, 16, 8, BF16, seed=60 + i).fill()
             for i, (lq, lk) in enumerate((([1400], [4000]), ([300], [5000]), ([200, 900, 77], [200, 950, 77])))]
    want = [c.prefill() for c in cases]
    for c, w in zip(cases, want):
        c.check(w)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(c.prefill())
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    outs = [torch.empty_like(w) for w in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, o in zip(cases, outs):
            c.prefill(out=o)
    for o in outs:
        o.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want)) and pkv.pkv_device_error() == 0


def many_short(seed, n, hq, hkv):
    rng = np.random.default_rng(seed)
    lq = [int(x) for x in rng.choice([0, 1, 5, 127, 128, 129, 200, 300], n)]
    return lq, [max(1, a + int(b)) for a, b in zip(lq, rng.integers(0, 900, n))]


@pytest.mark.parametrize("n,hq,hkv,dtype", [(40, 16, 8, BF16), (40, 32, 8, F16), (256, 4, 2, BF16), (70, 24, 4, F16)])
def test_many_short_tiles(pkv, n, hq, hkv, dtype):
    """Several units to a CTA (over 4 rounds of tiles), of one to ten key tiles; the same with an output that the
    32-byte stores can't take, which goes to the kernel of one tile to a CTA: the same bits."""
    c = Prefill(pkv, *many_short(n, n, hq, hkv), hq, hkv, dtype, seed=80 + n, extra_rows=3).fill()
    flat = torch.full((c.q.shape[0] * hq * 128 + 8,), 3.0, dtype=dtype, device="cuda")
    out, shifted = torch.full(c.q.shape, 3.0, dtype=dtype, device="cuda"), flat[8:].view(c.q.shape)
    c.prefill(out=out)
    c.check(out)
    assert bool((out[c.total:] == 3.0).all())
    c.prefill(out=shifted)
    assert shifted.data_ptr() % 32 == 16 and torch.equal(shifted, out)
    again = c.prefill(plan=pkv.pkv_prefill_plan(c.cq, c.ck))
    assert torch.equal(again[:c.total], out[:c.total]) and pkv.pkv_device_error() == 0


def test_many_short_tiles_nan_bad_blocks_and_lengths(pkv):
    lq, lk = many_short(3, 60, 16, 8)
    lq[7], lk[7] = 200, 700
    lq[20], lk[20] = 300, 600
    c = Prefill(pkv, lq, lk, 16, 8, BF16, seed=90).fill()
    want = c.prefill()
    c.v[c.first[7] + 650, 3, 100] = float("nan")
    out = c.fill().prefill()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[c.cq[7] + 150:c.cq[8], 6:8, 96:128] = True
    assert bool(out[hit].isnan().all()) and torch.equal(out[~hit], want[~hit])
    assert pkv.pkv_device_error() == 0
    c.tables[20, 1] = -7
    out = c.prefill()
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_BLOCK
    hit[c.cq[20]:c.cq[21]] = True
    assert torch.equal(out[~hit], want[~hit])
    c.tables[20, 1] = c.tables[20, 0]
    mark = torch.full_like(want, 7.0)
    c.f("pkv_prefill_varlen_q4")(c.q, c.d_cq, c.d_ck, 299, max(lk), c.scale, c.kc, c.vc, c.tables, out=mark)
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN   # the sequences of 300 are skipped
    long = torch.zeros_like(hit)
    for b, n in enumerate(lq):
        if n == 300:
            long[c.cq[b]:c.cq[b + 1]] = True
    assert bool((mark[long] == 7.0).all()) and torch.equal(mark[~long & ~hit], want[~long & ~hit])


def test_growing_logits(pkv):
    """The running maximum moves in every key tile."""
    c = Prefill(pkv, [400], [1500], 16, 8, BF16, seed=28)
    c.k = (c.k.float() + torch.linspace(-3, 3, 1500, device="cuda")[:, None, None]).to(BF16)
    c.q = c.q.abs()
    c.check(c.fill().prefill())


@pytest.mark.parametrize("max_q", [400, 2 ** 31 - 1])
def test_upper_bounds_of_the_lengths(pkv, max_q):
    """max_seqlen_q and max_seqlen_k may be any upper bounds."""
    c = Prefill(pkv, [200, 3], [300, 3], 4, 2, F16, seed=29).fill()
    want = c.prefill()
    c.check(want)
    out = c.f("pkv_prefill_varlen_q4")(c.q, c.d_cq, c.d_ck, max_q, 2 ** 31 - 1, c.scale, c.kc, c.vc, c.tables)
    assert torch.equal(out, want) and pkv.pkv_device_error() == 0


def test_shared_prefix_blocks(pkv):
    """Sequences that read the same physical blocks for their prefix."""
    c = Prefill(pkv, [60, 100, 200], [572, 612, 712], 16, 8, BF16, seed=22)
    c.tables[1:, :2] = c.tables[0, :2]
    for b in (1, 2):
        c.k[c.first[b]:c.first[b] + 512] = c.k[:512]
        c.v[c.first[b]:c.first[b] + 512] = c.v[:512]
    t = c.tables.cpu().numpy()
    p = [np.arange(n) for n in c.lens]
    slots = np.concatenate([t[b, x // 256] * 256 + x % 256 for b, x in enumerate(p)]).astype(np.int32)
    for b in (1, 2):
        slots[c.first[b]:c.first[b] + 512] = -1       # stored once, by the first sequence
    c.slots = torch.from_numpy(slots).cuda()
    c.fill()
    c.check(c.prefill())


def test_rows_behind_the_last_sequence_stay(pkv):
    c = Prefill(pkv, [40, 100], [40, 300], 16, 8, BF16, seed=23, extra_rows=37).fill()
    out = torch.full((c.total + 37, 16, 128), 5.0, dtype=BF16, device="cuda")
    assert c.prefill(out=out) is out
    c.check(out)
    assert bool((out[c.total:] == 5).all())


def test_nan_values_stay_behind_the_mask(pkv):
    """A NaN in V or K at a position reaches the rows that may attend to it, and only its group (V)."""
    c = Prefill(pkv, [200, 50], [330, 50], 16, 8, BF16, seed=24)
    c.v[300, 2, 40] = float("nan")                     # query rows 170.. of sequence 0, kv head 2, group 1
    c.k[310, 5, 0] = float("inf")                      # rows 180.., kv head 5: everything
    out = c.fill().prefill()
    assert c.pkv.pkv_device_error() == 0
    want = torch.zeros((250, 16, 128), dtype=torch.bool, device="cuda")
    want[170:200, 4:6, 32:64] = True
    want[180:200, 10:12] = True
    assert torch.equal(torch.isnan(out), want)
    c.check(out, {1})


def test_bad_blocks_and_lengths_are_reported(pkv):
    c = Prefill(pkv, [100, 100], [400, 400], 16, 8, BF16, seed=25).fill()
    good = c.tables.clone()
    c.tables[0, 1] = -7
    out = c.prefill()
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_BLOCK
    c.tables.copy_(good)
    c.check(out, {1})
    c.d_ck[2] = 450                                    # sequence 1: 50 keys for 100 query rows
    out = c.prefill()
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN
    c.d_ck[2] = 800
    c.check(c.prefill())
    plan = torch.tensor([(0 << 16) | 9], dtype=torch.int32, device="cuda")      # a sequence that is not there
    c.prefill(plan=plan)
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN


def test_store_prefill_decode_run(pkv):
    """The calls together as an engine makes them: two chunks of a prompt stored and attended to, then decode steps
    in a captured graph, over one 4-bit cache; every output against 64 bits over the values it stands for."""
    n0, n1, steps = 300, 229, 6
    c = Prefill(pkv, [n0], [n0 + n1 + steps], 16, 8, BF16, seed=26)
    total = n0 + n1
    kv = lambda a, b: (c.k[a:b], c.v[a:b], c.kc, c.vc, c.slots[a:b])  # noqa: E731
    q = W.normal_bf16((total + steps, 16, 128), W.make_generator(27, "cuda"), "cuda")
    kd, vd = R.dequantised(c.k), R.dequantised(c.v)
    half = torch.finfo(BF16).eps / 2

    def near(out, rows, first, rounding):
        ref = R.attention(q[rows], kd[:first + out.shape[0]], vd[:first + out.shape[0]], first, c.scale)
        big = float(vd.abs().amax())
        err = (out.double() - ref).abs()
        assert bool((err <= half * ref.abs() + big * rounding).all()), float(err.max())

    for a, b in ((0, n0), (n0, total)):
        pkv.pkv_store_kvcache_q4(*kv(a, b))
        cq, ck = torch.tensor([0, b - a], dtype=torch.int32), torch.tensor([0, b], dtype=torch.int32)
        out = pkv.pkv_prefill_varlen_q4(q[a:b], cq.cuda(), ck.cuda(), b - a, b, c.scale, c.kc, c.vc, c.tables)
        # k, v and p each rounded to bf16 (k moves a logit by half a step of the sum of its magnitudes, below 16 here)
        near(out, slice(a, b), a, half * (2 + 2 * 16) + 2.0 ** -16)
    qb, kb, vb = (torch.zeros((2, h, 128), dtype=BF16, device="cuda") for h in (16, 8, 8))
    slot = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
    tables = torch.cat((c.tables, torch.full_like(c.tables, -1)))
    ws = pkv.decode_q4_workspace(2, 4096)
    out = torch.empty((2, 16, 128), dtype=BF16, device="cuda")

    def step():
        pkv.pkv_store_decode_q4(qb, kb, vb, slot, c.kc, c.vc, tables, ctx, 4096, c.scale, ws, out=out)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(total, total + steps):
        qb[0], kb[0], vb[0] = q[i], c.k[i], c.v[i]
        slot[0], ctx[0] = c.slots[i], i + 1
        g.replay()
        near(out[:1], slice(i, i + 1), i, 2.0 ** -11 + 2.0 ** -14)
        assert not bool(out[1].any())
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("hkv", [4096, 1])
def test_most_heads(pkv, hkv):
    c = Prefill(pkv, [3, 130], [10, 300], 8192, hkv, BF16, seed=95).fill()
    c.check(c.prefill())


def test_most_sequences(pkv):
    n = 65535
    c = Prefill(pkv, [1] * n, [1 + i % 3 for i in range(n)], 2, 1, BF16, seed=96).fill()
    c.check(c.prefill(), set(range(0, n, 1997)) | {n - 1})
