"""Fused steps over the 4-bit cache in which every fetched tile takes a new row, one after the other in the same stage."""
import pytest
import torch

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


@pytest.mark.parametrize("lens,hq,hkv,dtype", [
    ([1 + i % 64 for i in range(760)], 16, 8, BF16),           # one unit an item, three to four items a warp
    ([1 + i % 16 for i in range(700)], 32, 8, F16),            # one tile; two pairs of heads share a kv head
    ([65 + 64 * (i % 3) for i in range(500)], 8, 8, BF16)])    # the new row alone in the item's last unit
def test_many_new_rows_in_one_stage(pkv, lens, hq, hkv, dtype):
    """Bytes and outputs are those of store then decode, call after call with other rows."""
    c = Case(pkv, lens, hq, hkv, dtype, seed=71).fill()
    B, gen = len(lens), W.make_generator(72, "cuda")
    slot = c.slots[torch.as_tensor(c.first[1:] - 1, device="cuda")]
    ws = c.workspace()
    for i in range(6):
        k, v = (W.normal((B, hkv, 128), gen, "cuda", dtype) * 2.0 ** (i - 2) for _ in range(2))
        kc, vc = c.kc.clone(), c.vc.clone()
        out = c.f("pkv_store_decode_q4")(c.q, k, v, slot, c.kc, c.vc, c.tables, c.ctx, c.max_ctx, c.scale, ws)
        c.f("pkv_store_kvcache_q4")(k, v, kc, vc, slot)
        assert torch.equal(c.kc, kc) and torch.equal(c.vc, vc)
        assert torch.equal(out, c.decode(ws))
    last = torch.as_tensor(c.first[1:] - 1, device="cuda")
    c.k[last], c.v[last] = k, v
    c.check(out, set(range(0, B, 37)))
