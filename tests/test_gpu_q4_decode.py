"""Decode over the 4-bit cache against attention in 64 bits over the values that
the stored tokens stand for, to a bound derived in q4_reference.decode_tolerance."""
import numpy as np
import pytest
import torch

import q4_reference as R
import workloads as W

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


class Case:
    """Sequences whose tokens are stored in a poisoned pool, block by block in shuffled order."""

    def __init__(self, pkv, lens, hq, hkv, dtype, seed=0, rows=None, spare=3):
        self.pkv, self.lens, self.hq, self.hkv, self.dtype = pkv, lens, hq, hkv, dtype
        gen, rng = W.make_generator(seed, "cuda"), np.random.default_rng(seed)
        total = sum(lens)
        if rows is None:
            self.k, self.v = (W.normal((total, hkv, 128), gen, "cuda", dtype) for _ in range(2))
        else:
            self.k, self.v = (x.to(dtype) for x in rows(total, gen))
        need = sum(-(-n // 256) for n in lens)
        order = rng.permutation(need + spare)
        width = max(1, -(-max(lens + [1]) // 256)) + 1
        tables = np.full((len(lens), width), -1, dtype=np.int32)
        slots, at = [], 0
        for b, n in enumerate(lens):
            nb = -(-n // 256)
            tables[b, :nb] = order[at:at + nb]
            at += nb
            p = np.arange(n)
            slots.append(tables[b, p // 256] * 256 + p % 256)
        self.slots = torch.from_numpy(np.concatenate(slots).astype(np.int32)).cuda()
        self.tables, self.ctx = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.kc, self.vc = (pkv.q4_cache(need + spare, hkv).fill_(0xff) for _ in range(2))
        qkv = W.normal((len(lens), (hq + 2 * hkv) * 128), gen, "cuda", dtype)
        self.q = qkv[:, :hq * 128].unflatten(1, (hq, 128))
        self.scale = W.SCALE
        self.max_ctx = max(lens + [1])
        self.first = np.concatenate(([0], np.cumsum(lens))).astype(int)

    def f(self, name):
        return getattr(self.pkv, name + ("_f16" if self.dtype == F16 else ""))

    def fill(self):
        self.f("pkv_store_kvcache_q4")(self.k, self.v, self.kc, self.vc, self.slots)
        return self

    def workspace(self, max_ctx=None):
        return self.pkv.decode_q4_workspace(len(self.lens), max_ctx or self.max_ctx, self.hq, self.hkv)

    def decode(self, ws=None, max_ctx=None, **kw):
        ws = self.workspace(max_ctx) if ws is None else ws
        return self.f("pkv_decode_q4")(self.q, self.kc, self.vc, self.tables, self.ctx, max_ctx or self.max_ctx,
                                       self.scale, ws, **kw)

    def check(self, out, only=None):
        assert self.pkv.pkv_device_error() == 0
        for b, n in enumerate(self.lens):
            if only is not None and b not in only:
                continue
            if n == 0:
                assert not bool(out[b].any()), f"row {b}: padding rows are zero"
                continue
            a, e = self.first[b], self.first[b + 1]
            ck, sk, zk = R.quantise(self.k[a:e])
            cv, sv, zv = R.quantise(self.v[a:e])
            k, v = R.values(ck, sk, zk), R.values(cv, sv, zv)
            q = self.q[b:b + 1]
            ref = R.attention(q, k, v, n - 1, self.scale)[0]
            tol = R.decode_tolerance(ref, q, k, v, cv, sv, zv, self.scale)
            err = (out[b].double() - ref).abs()
            assert bool((err <= tol).all()), \
                f"row {b} (context {n}): off by {float((err / tol).max()):.2f} of the bound, {float(err.max()):.3e}"


EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 255, 256, 257, 0, 300, 511, 512, 513, 1000]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv", [(16, 8), (8, 8), (32, 8), (8, 1), (12, 2), (1, 1), (10, 5)])
def test_edge_lengths(pkv, hq, hkv, dtype):
    c = Case(pkv, EDGES, hq, hkv, dtype, seed=hq).fill()
    c.check(c.decode())


@pytest.mark.parametrize("lens,hq,hkv,dtype", [
    ([1], 16, 8, BF16), ([1], 2, 1, F16), ([33], 16, 8, BF16), ([4096], 16, 8, BF16),
    ([40007], 32, 8, BF16),                       # many chunks: merged in groups, then the groups
    ([150001], 2, 1, F16),                        # over 4000 units of one head: several items per warp
    ([9001, 70000, 5], 16, 8, F16)])
def test_few_long_sequences(pkv, lens, hq, hkv, dtype):
    c = Case(pkv, lens, hq, hkv, dtype, seed=len(lens)).fill()
    c.check(c.decode())


def test_batches(pkv):
    """256 sequences (several items per warp, taken from the counter); sampled rows."""
    rng = np.random.default_rng(7)
    c = Case(pkv, rng.integers(512, 4097, 256).tolist(), 16, 8, BF16, seed=7).fill()
    ws = c.workspace(4096)
    out = c.decode(ws, 4096)
    c.check(out, set(range(0, 256, 13)))
    again = c.decode(ws, 4096)
    assert torch.equal(out, again)


def test_more_sequences_than_one_launch_takes(pkv):
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 300, 2500).tolist()
    c = Case(pkv, lens, 4, 2, F16, seed=8).fill()
    c.check(c.decode(), set(range(0, 2500, 61)) | {1023, 1024, 1025, 2047, 2048, 2499})


def scaled_rows(kind):
    def make(n, gen):
        k, v = (torch.randn((n, 2, 128), generator=gen, device="cuda") for _ in range(2))
        row = torch.exp2(torch.randint(-14, 9, (n, 2, 1), generator=gen, device="cuda").float())
        if kind == "offset":                       # keys far from zero, as channels with a bias have
            return k + 30.0, v - 12.0
        if kind == "tiny_v":
            return k, v * 2.0 ** -13
        if kind == "mixed_v":                      # rows of very different sizes next to one another
            return k, v * row
        if kind == "mixed_k":
            return k * row.clamp(max=4.0), v
        if kind == "constant":                     # scales of 0
            return k, torch.ones_like(v) * 0.75
        if kind == "growing":                      # the maximum moves in almost every unit
            return k + torch.linspace(0, 24, n, device="cuda")[:, None, None] * 0.1, v
        raise ValueError(kind)
    return make


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("kind", ["offset", "tiny_v", "mixed_v", "mixed_k", "constant", "growing"])
def test_value_distributions(pkv, kind, dtype):
    c = Case(pkv, [1, 40, 700, 3000], 4, 2, dtype, seed=3, rows=scaled_rows(kind)).fill()
    if kind == "growing":
        c.q = c.q.abs()
    c.check(c.decode())


@pytest.mark.parametrize("factor", [2.0 ** -20, 2.0 ** -6, 2.0 ** 5])
def test_query_sizes(pkv, factor):
    c = Case(pkv, [5, 300, 1111], 16, 8, BF16, seed=4).fill()
    c.q = c.q * factor
    c.q[1, 3] = 0                                   # a head of zeros: plain averages
    c.q[2, ::2] *= 2.0 ** -10                       # heads of a pair scaled differently
    c.check(c.decode())


@pytest.mark.parametrize("power", [100, 113, 114, 120, 126])
def test_queries_near_the_end_of_bf16(pkv, power):
    """Logits of up to 2^128 in fp32: the largest takes all the weight. The bound is the output's rounding and that of
    p s to fp16 (p = 1): half a step each of the largest value, and fp32 terms far below them."""
    c = Case(pkv, [5, 300, 1111], 4, 2, BF16, seed=5)
    c.k *= 2.0 ** -4
    c.fill()
    c.q = c.q.sign() * 2.0 ** power
    c.q[1] *= 1.5
    out = c.decode().double()
    assert pkv.pkv_device_error() == 0
    for b in range(3):
        a, e = c.first[b], c.first[b + 1]
        k, v = (R.values(*R.quantise(x[a:e])) for x in (c.k, c.v))
        for h in range(4):
            logits = k[:, h // 2] @ c.q[b, h].double()
            best = logits.topk(2).values
            assert float(best[0] - best[1]) > 2.0 ** -16 * float(logits.abs().max()), "inputs: a clear largest logit"
            want = v[int(logits.argmax()), h // 2]
            tol = (2.0 ** -8 + 2.0 ** -10) * want.abs().max()
            assert bool(((out[b, h] - want).abs() <= tol).all()), (b, h)


def test_nan_rows_reach_only_their_sequence_and_group(pkv):
    c = Case(pkv, [100, 100, 100], 4, 2, BF16, seed=5)
    c.v[50, 0, 40] = float("nan")                   # sequence 0, kv head 0, group 1 of V
    c.k[150, 1, 0] = float("inf")                   # sequence 1, kv head 1: every logit of that head's row
    out = c.fill().decode()
    assert c.pkv.pkv_device_error() == 0
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[0, 0:2, 32:64] = True
    want[1, 2:4] = True
    assert torch.equal(nan, want)
    c.check(out, {2})


def test_queries_strided_and_out_given(pkv):
    c = Case(pkv, [77, 500], 16, 8, BF16, seed=6).fill()
    out = torch.full((2, 16, 128), 9.0, dtype=BF16, device="cuda")
    assert c.decode(out=out) is out
    c.check(out)
    assert torch.equal(out, c.f("pkv_decode_q4")(c.q.contiguous(), c.kc, c.vc, c.tables, c.ctx, c.max_ctx, c.scale,
                                                 c.workspace()))


def test_one_workspace_for_calls_of_other_sizes(pkv):
    """A workspace of the largest call serves calls of any sizes and head counts in between."""
    big = Case(pkv, [3000] * 40, 4, 2, F16, seed=9).fill()
    few = Case(pkv, [9000], 16, 4, BF16, seed=10).fill()
    many = Case(pkv, list(range(0, 900)), 2, 2, BF16, seed=11).fill()
    ws = torch.zeros(max(c.workspace().numel() for c in (big, few, many)), dtype=torch.uint8, device="cuda")
    want = [c.decode() for c in (big, few, many)]
    for c, w in list(zip((big, few, many), want)) * 2 + [(few, want[1]), (big, want[0])]:
        assert torch.equal(c.decode(ws), w)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv", [(16, 8), (32, 8), (3, 3)])
def test_step_is_store_then_decode(pkv, hq, hkv, dtype):
    """The fused step's bytes and output are those of the two calls; padding rows and rows without a new token too."""
    lens = [1, 16, 17, 0, 256, 257, 700, 33, 2000, 32]
    c = Case(pkv, lens, hq, hkv, dtype, seed=12)
    last = torch.tensor([c.first[b + 1] - 1 for b, n in enumerate(lens) if n], device="cuda")
    B = len(lens)
    slot = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    new = torch.zeros((2, B, hkv, 128), dtype=dtype, device="cuda")
    live = torch.tensor([b for b, n in enumerate(lens) if n], device="cuda")
    slot[live] = c.slots[last]
    new[0, live], new[1, live] = c.k[last], c.v[last]
    c.fill()                                        # everything stored already ...
    slot[7] = -1                                    # (sequence 7 keeps its stored token)
    kc, vc = c.kc.clone(), c.vc.clone()
    poison = torch.randn((B, hkv, 128), device="cuda").to(dtype)
    c.f("pkv_store_kvcache_q4")(poison, poison, c.kc, c.vc, slot)      # ... then the last tokens overwritten
    out = c.f("pkv_store_decode_q4")(c.q, new[0], new[1], slot, c.kc, c.vc, c.tables, c.ctx, c.max_ctx, c.scale,
                                     c.workspace())
    assert torch.equal(c.kc, kc) and torch.equal(c.vc, vc)
    assert torch.equal(out, c.decode())
    c.check(out)


def test_step_wrong_slots_are_not_stored(pkv):
    c = Case(pkv, [40, 300], 4, 2, BF16, seed=13).fill()
    kc = c.kc.clone()
    rows = torch.zeros((2, 2, 128), dtype=BF16, device="cuda")
    slot = torch.tensor([int(c.slots[3]), 10 ** 6], dtype=torch.int32, device="cuda")
    out = c.f("pkv_store_decode_q4")(c.q, rows, rows, slot, c.kc, c.vc, c.tables, c.ctx, c.max_ctx, c.scale,
                                     c.workspace())
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SLOT
    assert torch.equal(c.kc, kc)
    c.check(out)


def test_step_slot_without_context(pkv):
    """A padding row has no position that a slot could belong to: nothing is stored, and the slot is reported."""
    for lens in ([40, 0], [40] + [0] * 40):         # either form of the item table
        c = Case(pkv, lens, 4, 2, BF16, seed=17).fill()
        kc = c.kc.clone()
        B = len(lens)
        rows = torch.zeros((B, 2, 128), dtype=BF16, device="cuda")
        slot = torch.full((B,), -1, dtype=torch.int32, device="cuda")
        step = lambda: c.f("pkv_store_decode_q4")(c.q, rows, rows, slot, c.kc, c.vc, c.tables, c.ctx, c.max_ctx,
                                                  c.scale, c.workspace())
        c.check(step())
        slot[1] = int(c.slots[3])
        out = step()
        assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SLOT
        assert torch.equal(c.kc, kc)
        c.check(out)


def test_bad_blocks_and_lengths_are_reported(pkv):
    c = Case(pkv, [300, 300, 300, 40], 4, 2, BF16, seed=14).fill()
    good = c.tables.clone()
    c.tables[1, 1] = 10 ** 6
    out = c.decode()
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_BLOCK
    c.tables.copy_(good)
    c.check(out, {0, 2, 3})
    ctx = c.ctx.clone()
    c.ctx[0], c.ctx[2] = -1, 301                    # negative; above max_context_len
    out = c.decode()
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN
    assert not bool(out[0].any()) and not bool(out[2].any())
    c.ctx[0], c.ctx[2] = 300, 2000                  # past the block table's width
    out = c.decode(max_ctx=4000)
    assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN
    assert not bool(out[2].any())
    c.ctx.copy_(ctx)
    c.check(c.decode(), None)


def test_graph_replays_follow_the_lengths(pkv):
    """One captured step replayed while the contexts grow, shrink and vanish; two graphs share the workspace in turn."""
    lens = [700, 40, 1, 1500, 256]
    c = Case(pkv, lens, 16, 8, BF16, seed=15).fill()
    ws = c.workspace(4096)
    out = torch.empty((5, 16, 128), dtype=BF16, device="cuda")
    out2 = torch.empty_like(out)
    c.decode(ws, 4096, out=out)
    torch.cuda.synchronize()
    graphs = []
    for o in (out, out2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.decode(ws, 4096, out=o)
        graphs.append(g)
    full = c.lens
    for now in ([700, 40, 1, 1500, 256], [0, 33, 1, 1024, 255], [0] * 5, [512, 0, 0, 1499, 3]):
        c.ctx.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(3.0)
        out2.fill_(4.0)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, out2)
        for b, n in enumerate(now):
            if n == 0:
                assert not bool(out[b].any())
        sub = Case.__new__(Case)
        sub.__dict__.update(c.__dict__)
        sub.lens = now
        sub.first = c.first.copy()
        for b, n in enumerate(now):                 # the first n tokens of each sequence
            if n:
                a = c.first[b]
                sub2 = Case.__new__(Case)
                sub2.__dict__.update(c.__dict__)
                sub2.lens, sub2.first, sub2.q = [n], np.array([a, a + n]), c.q[b:b + 1]
                sub2.check(out[b:b + 1])
    assert c.lens is full


def test_another_stream(pkv):
    c = Case(pkv, [300, 2000], 16, 8, F16, seed=16)
    s = torch.cuda.Stream()
    ws = c.workspace()
    s.wait_stream(torch.cuda.current_stream())
    c.f("pkv_store_kvcache_q4")(c.k, c.v, c.kc, c.vc, c.slots, stream=s)
    out = torch.empty((2, 16, 128), dtype=F16, device="cuda")
    c.decode(ws, out=out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    c.check(out)


def test_calls_at_once(pkv):
    """Two streams, a workspace each."""
    cases = [Case(pkv, [700, 40, 3000], 16, 8, BF16, seed=18).fill(), Case(pkv, [9000, 1], 32, 8, F16, seed=19).fill()]
    spaces = [c.workspace() for c in cases]
    want = [c.decode(w) for c, w in zip(cases, spaces)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for c, s, w in zip(cases, streams, spaces):
            with torch.cuda.stream(s):
                got.append(c.decode(w))
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    for c, w in zip(cases, want):
        c.check(w)


def test_cache_past_32_bit_offsets(pkv):
    """Block ids whose byte offsets pass 2^32, for K and V."""
    spare = 2 ** 32 // (8 * 20480) + 2
    c = Case(pkv, [700, 33], 16, 8, BF16, seed=17, spare=spare)
    ids = torch.arange(c.kc.shape[0] - 4, c.kc.shape[0], dtype=torch.int32)
    c.tables[0, :3], c.tables[1, 0] = ids[:3].cuda(), int(ids[3])
    t = c.tables.cpu().numpy()
    p = [np.arange(n) for n in c.lens]
    c.slots = torch.from_numpy(np.concatenate([t[b, x // 256] * 256 + x % 256 for b, x in enumerate(p)])
                               .astype(np.int32)).cuda()
    c.fill()
    c.check(c.decode())


@pytest.mark.parametrize("hkv", [8192, 4])
def test_most_heads(pkv, hkv):
    c = Case(pkv, [10, 300 if hkv == 4 else 33], 8192, hkv, F16, seed=95, spare=1).fill()
    c.check(c.decode())


def test_most_sequences(pkv):
    n = 65535
    c = Case(pkv, [i % 3 for i in range(n)], 2, 1, BF16, seed=96).fill()
    c.check(c.decode(), set(range(0, n, 1997)) | {n - 1, n - 2, n - 3})
