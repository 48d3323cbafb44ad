"""The 4-bit calls where their kernels change over: batches around the sequences that one launch takes, and more rows
than one grid dimension."""
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


def test_batches_around_one_launch(pkv):
    """2500 sequences in launches of 768: every row as in calls of a launch's sequences alone, and the rows beside the
    launches' borders against 64 bits."""
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 300, 2500).tolist()
    for b in (767, 768, 1535, 1536, 2303, 2304, 2499):
        lens[b] = 200 + b % 100
    c = Case(pkv, lens, 4, 2, F16, seed=8).fill()
    out = c.decode()
    c.check(out, {0, 767, 768, 1535, 1536, 2303, 2304, 2499})
    ws = pkv.decode_q4_workspace(768, c.max_ctx, 4, 2)
    for a in range(0, 2500, 768):
        part = pkv.pkv_decode_q4_f16(c.q[a:a + 768], c.kc, c.vc, c.tables[a:a + 768].contiguous(),
                                     c.ctx[a:a + 768].contiguous(), c.max_ctx, c.scale, ws)
        assert torch.equal(part, out[a:a + 768])
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("n", [767, 768, 769, 1536, 1537])
def test_steps_around_one_launch(pkv, n):
    """The fused step of every row, padding rows among them."""
    lens = [0 if i % 11 == 5 else 1 + i * 7 % 90 for i in range(n)]
    c = Case(pkv, lens, 2, 1, BF16, seed=n).fill()
    gen = W.make_generator(n, "cuda")
    k, v = (W.normal_bf16((n, 1, 128), gen, "cuda") for _ in range(2))
    live = torch.tensor([x > 0 for x in lens], device="cuda")
    last = torch.as_tensor(np.maximum(c.first[1:] - 1, 0), device="cuda")
    slot = torch.where(live, c.slots[last], torch.full_like(c.slots[last], -1))
    kc, vc = c.kc.clone(), c.vc.clone()
    ws = c.workspace()
    out = pkv.pkv_store_decode_q4(c.q, k, v, slot, c.kc, c.vc, c.tables, c.ctx, c.max_ctx, c.scale, ws)
    pkv.pkv_store_kvcache_q4(k, v, kc, vc, slot)
    assert torch.equal(c.kc, kc) and torch.equal(c.vc, vc) and torch.equal(out, c.decode(ws))
    c.k[last[live]], c.v[last[live]] = k[live], v[live]
    c.check(out, {0, n // 2, n - 2, n - 1} | set(range(760, min(n, 772))))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_past_one_grid_dimension(pkv, dtype):
    """Over 65535 x 32 rows in one call (a block of the kernels takes 32): written and read back, those in the grid's
    third dimension among them, and a row of slot -1 on either side of it."""
    n = 65535 * 32 + 4097
    gen = W.make_generator(6, "cuda")
    k, v = (W.normal((n, 1, 128), gen, "cuda", dtype) for _ in range(2))
    kc, vc = (pkv.q4_cache(-(-n // 256), 1).fill_(0xff) for _ in range(2))
    slots = torch.arange(n, dtype=torch.int32, device="cuda").flip(0)
    dead = torch.tensor([5, 65535 * 32 - 1, 65535 * 32 + 1, n - 1], device="cuda")
    slots[dead] = -1
    f16 = dtype == F16
    (pkv.pkv_store_kvcache_q4_f16 if f16 else pkv.pkv_store_kvcache_q4)(k, v, kc, vc, slots)
    got = (pkv.pkv_load_kvcache_q4_f16 if f16 else pkv.pkv_load_kvcache_q4)(kc, vc, slots)
    half = torch.finfo(dtype).eps / 2
    for g, x in zip(got, (k, v)):
        assert not bool(g[dead].any())
        for a in list(range(0, n, 65536 * 8)) + [65535 * 32]:      # in parts, to bound the 64-bit copies
            e = min(n, a + 65536 * 8)
            live = slots[a:e] >= 0
            ref = R.dequantised(x[a:e][live])
            assert bool(((g[a:e][live].double() - ref).abs() <= ref.abs() * (half + 2.0 ** -23) + 2.0 ** -25).all())
    for cache in (kc, vc):                                          # the cells of the rows that were left out
        for s in (n - 1 - dead).tolist():
            cell = cache[s // 256, 0, s % 256 // 16]
            assert bool((cell[s % 16 * 64:s % 16 * 64 + 64] == 0xff).all())
            assert bool((cell[1024 + s % 16 * 16:1024 + s % 16 * 16 + 16] == 0xff).all())
    assert pkv.pkv_device_error() == 0
