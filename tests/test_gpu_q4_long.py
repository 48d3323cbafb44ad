"""Decode of sequences of many chunks over the 4-bit cache, to a bound that a lost or misweighted chunk would pass."""
import pytest
import torch

import q4_long_reference as L
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


@pytest.mark.parametrize("spread", [0.0, 0.6])
@pytest.mark.parametrize("lens,hq,hkv,dtype", [
    ([40007], 32, 8, BF16),                          # over 100 chunks: joined in groups of 16, then the groups
    ([150001], 2, 1, F16),                           # several items a warp, taken from the counter
    ([300007], 1, 1, BF16),                          # one head to an item
    ([9001, 70000, 513], 16, 8, F16),
    ([20000 + 1111 * i for i in range(40)], 8, 1, BF16)])  # more than 32 sequences: the other form of the item table
def test_long_sequences(pkv, lens, hq, hkv, dtype, spread):
    c = Case(pkv, lens, hq, hkv, dtype, seed=len(lens) + hq, rows=L.rows(hkv, spread)).fill()
    ws = c.workspace()
    out = c.decode(ws)
    for b in range(0, len(lens), 7):
        a, e = c.first[b], c.first[b + 1]
        ref, tol = L.reference(c.q[b:b + 1], c.k[a:e], c.v[a:e], c.scale)
        err = (out[b].double() - ref).abs()
        assert bool((err <= tol).all()), f"row {b}: off by {float((err / tol).max()):.2f} of the bound"
    for _ in range(3):
        assert torch.equal(c.decode(ws), out)
    assert pkv.pkv_device_error() == 0
