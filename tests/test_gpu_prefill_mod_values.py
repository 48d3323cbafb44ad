"""Prefill with modified scores over values that are not finite and long ranges of keys: they reach the rows that see their
key, in their dim, and nothing else is lost by them."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


def _rows(seqs, hq, hkv, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lq, lk = sum(n for _, n in seqs), sum(c + n for c, n in seqs)
    return [torch.randn((n, h, D), generator=g, device="cuda").to(dtype) for n, h in ((lq, hq), (lk, hkv), (lk, hkv))]


def _run(pkv, q, k, v, seqs, **mods):
    fn = pkv.pkv_prefill_varlen_mod_f16 if q.dtype == torch.float16 else pkv.pkv_prefill_varlen_mod
    cu_q, cu_k = [0], [0]
    for c, n in seqs:
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + c + n)
    cu = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu_q, cu_k)]
    return fn(q, *cu, max(n for _, n in seqs), max(c + n for c, n in seqs), D ** -0.5, k=k, v=v, **mods)


def _near(a, b, v, where):
    """Rows that are computed again do not round p: half a step of 16 bits of sum p |v| apart, and either result rounded."""
    eps = torch.finfo(a.dtype).eps
    room = eps * (b.float().abs() + float(v.float().abs().nan_to_num(0, 0, 0).max()))
    return bool(((a.float() - b.float()).abs() <= room)[where].all())


@pytest.mark.parametrize("dtype,value", [(torch.bfloat16, float("nan")), (torch.float16, float("inf"))])
def test_one_bad_value_before_a_long_range(pkv, dtype, value):
    """Whole items and split ones, and another sequence behind them. Rows of the first and of the last tile do not see a
    value that their tile's products take in."""
    cached, new = 45000, 12800
    seqs = [(cached, new), (0, 200)]
    q, k, v = _rows(seqs, 2, 1, dtype)
    clean = _run(pkv, q, k, v, seqs)
    v[cached + 127, 0, 5] = value
    v[cached + new - 1, 0, 77] = value
    out = _run(pkv, q, k, v, seqs)
    assert pkv.pkv_device_error() == 0
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[127:new, :, 5] = True
    bad[new - 1, :, 77] = True
    assert torch.equal(~torch.isfinite(out), bad)
    assert _near(out, clean, v, ~bad)
