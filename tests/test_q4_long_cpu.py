"""That the bound of q4_long_reference accepts what the kernel rounds and nothing that has lost a part of the sequence."""
import pytest
import torch

import q4_long_reference as L
import q4_reference as R

SCALE = 128 ** -0.5


def inputs(n, hq, hkv, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    k, v = (x.to(dtype) for x in L.rows(hkv)(n, gen))
    return torch.randn((1, hq, 128), generator=gen).to(dtype), k, v


@pytest.mark.parametrize("n,hq,hkv,dtype,chunk", [
    (60001, 2, 1, torch.float16, 1344), (20007, 2, 1, torch.bfloat16, 384), (30000, 2, 2, torch.float16, 2048)])
def test_bound(n, hq, hkv, dtype, chunk):
    q, k, v = inputs(n, hq, hkv, dtype, n)
    ref, tol = L.reference(q, k, v, SCALE)
    chunks = -(-n // chunk)

    def accepted(x):
        return bool(((x - ref).abs() <= tol).all())

    assert accepted(L.as_the_kernel_rounds(q, k, v, SCALE, chunk))
    assert not accepted(torch.zeros_like(ref))
    for i in {0, 15, 16, chunks // 2, chunks - 1}:            # the merge takes 16 chunks at a time
        if i < chunks:
            assert not accepted(L.as_the_kernel_rounds(q, k, v, SCALE, chunk, lost=(i,))), i
            if i < chunks - 1:
                assert not accepted(L.as_the_kernel_rounds(q, k, v, SCALE, chunk, off=(i,))), i
    assert not accepted(L.as_the_kernel_rounds(q, k, v, SCALE, chunk, lost=range(0, min(16, chunks - 1))))


def test_bound_with_chunks_of_other_maxima():
    gen = torch.Generator().manual_seed(5)
    k, v = (x.to(torch.bfloat16) for x in L.rows(1, 0.6)(20000, gen))
    q = torch.randn((1, 2, 128), generator=gen).to(torch.bfloat16)
    ref, tol = L.reference(q, k, v, SCALE)
    assert bool(((L.as_the_kernel_rounds(q, k, v, SCALE, 512) - ref).abs() <= tol).all())
    assert not bool((ref.abs() <= tol).all())
