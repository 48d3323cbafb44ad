"""A tile plan over the 4-bit cache names exactly the tiles that a call computes, whichever form of the kernel takes it."""
import numpy as np
import pytest
import torch

from test_gpu_q4_prefill import Prefill, many_short

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


def rows_of(c, plan):
    """Which rows the plan's items hold."""
    hit = torch.zeros(c.q.shape[0], dtype=torch.bool, device="cuda")
    for code in plan.tolist():
        qt, b = code >> 16, code & 0xffff
        hit[c.cq[b] + 128 * qt:min(c.cq[b] + 128 * (qt + 1), c.cq[b + 1])] = True
    return hit


CASES = [
    (many_short(40, 70, 16, 8), 32, 8, BF16),          # several units to a CTA
    (many_short(41, 256, 16, 8), 16, 8, F16),
    (([700, 300, 1300], [2000, 300, 1300]), 16, 8, BF16),    # a tile to a CTA
    (([300, 200], [5000, 4000]), 16, 8, F16)]          # keys split over CTAs


@pytest.mark.parametrize("lens,hq,hkv,dtype", CASES)
def test_a_plan_in_two_calls(pkv, lens, hq, hkv, dtype):
    """Every second item, then the others: each call writes its own tiles' rows and no other."""
    c = Prefill(pkv, *lens, hq, hkv, dtype, seed=len(lens[0]), extra_rows=2).fill()
    want = c.prefill()
    c.check(want)
    plan = pkv.pkv_prefill_plan(c.cq, c.ck)
    halves = [plan[::2].contiguous(), plan[1::2].contiguous()]
    out = torch.full_like(want, 3.0)
    for half in halves:
        before = out.clone()
        c.prefill(out=out, plan=half)
        hit = rows_of(c, half)
        assert bool(hit.any()) and torch.equal(out[~hit], before[~hit])
        assert not bool((out[hit] == 3.0).all((1, 2)).any())
    assert bool((out[c.total:] == 3.0).all())
    c.check(out)
    assert pkv.pkv_device_error() == 0


def test_stale_items(pkv):
    """Items past a sequence's end are skipped; items of sequences that are not there are skipped and reported. The plan
    is long enough for several units to a CTA."""
    c = Prefill(pkv, *many_short(42, 120, 16, 8), 16, 8, BF16, seed=5).fill()
    want = c.prefill()
    plan = pkv.pkv_prefill_plan(c.cq, c.ck)
    past = torch.tensor([(n // 128 + 1 + 40 * i) << 16 | b for b, n in enumerate(c.lq[:60]) for i in (0, 1)],
                        dtype=torch.int32, device="cuda")
    mixed = torch.cat((past[:50], plan, past[50:]))[torch.from_numpy(np.random.default_rng(6).permutation(120 + len(plan))).cuda()]
    assert mixed.numel() * 8 >= 4 * 152
    out = torch.full_like(want, 3.0)
    c.prefill(out=out, plan=mixed.contiguous())
    assert pkv.pkv_device_error() == 0 and torch.equal(out, want)
    for strange in (3 << 16 | 120, 65535, 32767 << 16 | 65535, -1 << 16 | 5):
        bad = torch.cat((mixed, torch.tensor([strange], dtype=torch.int32, device="cuda")))
        out.fill_(3.0)
        c.prefill(out=out, plan=bad)
        assert pkv.pkv_device_error() == pkv.PKV_DEVERR_BAD_SEQLEN and torch.equal(out, want)


def test_a_plan_of_more_items_than_the_units_list_holds(pkv):
    """The same tiles named more than once: each is computed, to the same rows."""
    c = Prefill(pkv, *many_short(43, 90, 4, 2), 4, 2, F16, seed=7).fill()
    want = c.prefill()
    plan = pkv.pkv_prefill_plan(c.cq, c.ck)
    for times in (4, 12):
        out = torch.full_like(want, 3.0)
        c.prefill(out=out, plan=plan.repeat(times))
        assert torch.equal(out, want)
    assert pkv.pkv_device_error() == 0
