"""A decode workspace that a call left marked after a wait ran out: later calls refuse it instead of joining partial
results that belong to that call. The mark is set from the host; no wait is made to run out."""
import pytest
import torch

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
    ([300, 0, 5], 16, 8, BF16), ([40007], 2, 1, F16), ([2000] * 300, 16, 8, BF16), ([40] * 1000, 4, 4, F16)])
def test_marked_workspace_is_refused_until_zeroed(pkv, lens, hq, hkv, dtype):
    c = Case(pkv, lens, hq, hkv, dtype, seed=81).fill()
    ws = c.workspace()
    want = c.decode(ws)
    words = ws[:8].view(torch.int32)                # {next item, warps done}
    assert words.tolist() == [0, 0]
    words[1] = -2 ** 31
    ws[8:2048] = 1                                  # tickets taken by only some of a sequence's chunks
    out = torch.full_like(want, 3.0)
    kc, vc = c.kc.clone(), c.vc.clone()
    B = len(lens)
    new = torch.ones((B, hkv, 128), dtype=dtype, device="cuda")
    slot = torch.full((B,), int(c.slots[lens[0] - 1]), dtype=torch.int32, device="cuda")
    for _ in range(2):
        c.decode(ws, out=out)
        assert pkv.pkv_device_error() == pkv.PKV_DEVERR_TIMEOUT
        c.f("pkv_store_decode_q4")(c.q, new, new, slot, c.kc, c.vc, c.tables, c.ctx, c.max_ctx, c.scale, ws, out=out)
        assert pkv.pkv_device_error() == pkv.PKV_DEVERR_TIMEOUT
        assert bool((out == 3.0).all()) and torch.equal(c.kc, kc) and torch.equal(c.vc, vc)
    ws.zero_()
    assert torch.equal(c.decode(ws, out=out), want) and torch.equal(c.decode(ws), want)
    assert pkv.pkv_device_error() == 0


def test_counters_are_zero_after_calls(pkv):
    """Counters and tickets of calls of several shapes, one after the other on one workspace: all zero again."""
    cases = [Case(pkv, [3000] * 60, 4, 2, F16, seed=82).fill(), Case(pkv, [50000, 7], 16, 4, BF16, seed=83).fill(),
             Case(pkv, list(range(0, 900)), 2, 2, BF16, seed=84).fill()]
    ws = torch.zeros(max(c.workspace().numel() for c in cases), dtype=torch.uint8, device="cuda")
    counters = ws[:256 + (ws.numel() // 128 & ~255)]
    for c in cases * 2:
        c.decode(ws)
        assert not bool(counters.any())
    assert pkv.pkv_device_error() == 0
