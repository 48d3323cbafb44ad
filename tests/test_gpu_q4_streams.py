"""The 4-bit calls on a stream of the caller's, beside work that the current stream is busy with: what they return
depends on nothing that happens there."""
import pytest
import torch

import q4_reference as R
import workloads as W
from test_gpu_q4_decode import Case
from test_gpu_q4_prefill import Prefill

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


class Busy:
    """A few milliseconds of ordinary work on the current stream."""

    def __init__(self):
        self.a = torch.randn((8192, 8192), device="cuda").to(BF16)

    def __call__(self):
        for _ in range(4):
            self.a @ self.a


@pytest.mark.parametrize("raw", [False, True])
def test_rows_read_back_on_another_stream(pkv, raw):
    """k and v made by the call: rows of live slots whole, rows of slot -1 zero, though the current stream is behind."""
    n = 16384
    gen = W.make_generator(31, "cuda")
    k, v = (W.normal_bf16((n, 8, 128), gen, "cuda") for _ in range(2))
    kc, vc = pkv.q4_cache(n // 256), pkv.q4_cache(n // 256)
    slots = torch.randperm(n, generator=gen, device="cuda").int()
    pkv.pkv_store_kvcache_q4(k, v, kc, vc, slots)
    dead = torch.arange(n, device="cuda") % 7 == 3
    slots[dead] = -1
    want = pkv.pkv_load_kvcache_q4(kc, vc, slots)
    for got, x in zip(want, (k, v)):                # half a step of bf16, and the fp32 rounding before it
        ref = R.dequantised(x[~dead])
        assert bool(((got[~dead].double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -25).all())
    assert not bool(want[0][dead].any()) and not bool(want[1][dead].any())
    busy, s = Busy(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        # memory that the allocator will hand out again holds something else than zeros
        junk = [torch.full((n, 8, 128), 9.0, dtype=BF16, device="cuda") for _ in range(2)]
        del junk
        busy()
        s.wait_stream(torch.cuda.current_stream())
        busy()
        got = pkv.pkv_load_kvcache_q4(kc, vc, slots, stream=s.cuda_stream if raw else s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert pkv.pkv_device_error() == 0


def test_attention_on_another_stream(pkv):
    """out made by the call, on memory that the current stream has just freed and still writes to."""
    d = Case(pkv, [700, 40, 3000], 16, 8, F16, seed=32).fill()
    p = Prefill(pkv, [300, 40], [900, 40], 16, 8, BF16, seed=33).fill()
    want_d, want_p, ws = d.decode(), p.prefill(), d.workspace()
    busy, s = Busy(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        s.wait_stream(torch.cuda.current_stream())
        busy()
        for shape in (want_d, want_p):
            junk = torch.empty_like(shape)
            junk.fill_(7.0)                          # queued behind the work above
            del junk
        got_d, got_p = d.decode(ws, stream=s), p.prefill(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got_d, want_d) and torch.equal(got_p, want_p)
    d.check(want_d)
    p.check(want_p)


def test_load_in_a_graph_forked_to_another_stream(pkv):
    """Captured: the fill and the gather are one branch of the graph."""
    n = 2000
    gen = W.make_generator(34, "cuda")
    k, v = (W.normal_bf16((n, 8, 128), gen, "cuda") for _ in range(2))
    kc, vc = pkv.q4_cache(8), pkv.q4_cache(8)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    pkv.pkv_store_kvcache_q4(k, v, kc, vc, slots)
    want = pkv.pkv_load_kvcache_q4(kc, vc, slots)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = pkv.pkv_load_kvcache_q4(kc, vc, slots, stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for t in got:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_raw_handles_of_the_default_streams(pkv):
    """0 and cudaStreamLegacy (1) are torch's default stream, 2 is the thread's own; tensors made by the call."""
    k = W.normal_bf16((300, 8, 128), W.make_generator(35, "cuda"), "cuda")
    kc, vc = pkv.q4_cache(2), pkv.q4_cache(2)
    slots = torch.arange(300, dtype=torch.int32, device="cuda")
    pkv.pkv_store_kvcache_q4(k, k, kc, vc, slots)
    want = pkv.pkv_load_kvcache_q4(kc, vc, slots)
    torch.cuda.synchronize()
    for handle in (0, 1, 2, torch.cuda.current_stream()):
        got = pkv.pkv_load_kvcache_q4(kc, vc, slots, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert pkv.pkv_device_error() == 0
