"""Where the binding of the 4-bit calls makes the tensors that it returns: on the stream that the call runs on. The GPU
is replaced by recorders, so the order of the steps can be checked without one."""
import contextlib

import pytest
import torch


class Recorder:
    def __init__(self, monkeypatch, m):
        self.steps, self.stream = [], "current"
        real = {name: getattr(torch, name) for name in ("zeros", "empty", "empty_like")}

        def maker(name):
            def make(*a, **kw):
                self.steps.append((name.removesuffix("_like"), self.stream))
                return real[name](*a, **kw)
            return make

        @contextlib.contextmanager
        def stream(s):
            before, self.stream = self.stream, s.cuda_stream
            yield
            self.stream = before

        class Stream:
            def __init__(self, handle, device=None):
                self.cuda_stream = handle

        self.Stream = Stream
        for name in real:
            monkeypatch.setattr(torch, name, maker(name))
        monkeypatch.setattr(torch.cuda, "Stream", Stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda: "here")
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.steps.append(("kept for", s)))
        monkeypatch.setattr(m, "_current_device", lambda: -1)       # the device of the CPU's tensors
        monkeypatch.setattr(m, "_current_raw_stream", lambda dev: "current")

    def entry(self, *args):
        self.steps.append(("launch", args[-1]))
        return 0


@pytest.fixture
def m():
    import paged_kv_cache_kvh_gb300 as pkv
    return pkv


def load(m, rec, **kw):
    cache = torch.zeros((2, 8, 16, 1280), dtype=torch.uint8)
    slots = torch.zeros(3, dtype=torch.int32)
    rec.steps.clear()
    return m._load_q4(rec.entry, torch.bfloat16, cache, cache, slots, kw.pop("k", None), kw.pop("v", None), **kw)


def decode(m, rec, **kw):
    cache, q = torch.zeros((2, 8, 16, 1280), dtype=torch.uint8), torch.zeros((2, 16, 128), dtype=torch.float16)
    i32 = torch.zeros((2, 2), dtype=torch.int32)
    ws = torch.zeros(64, dtype=torch.uint8)
    rec.steps.clear()
    return m._decode_q4(rec.entry, torch.float16, q, None, cache, cache, i32, i32[0], 512, 0.1, ws, None, **kw)


def prefill(m, rec, **kw):
    cache, q = torch.zeros((2, 8, 16, 1280), dtype=torch.uint8), torch.zeros((2, 16, 128), dtype=torch.bfloat16)
    i32 = torch.zeros((2, 2), dtype=torch.int32)
    rec.steps.clear()
    return m._prefill_q4(rec.entry, torch.bfloat16, q, i32[0], i32[0], 1, 1, 0.1, cache, cache, i32, None, None, **kw)


@pytest.mark.parametrize("call", [load, decode, prefill])
def test_returned_tensors_are_made_on_the_calls_stream(monkeypatch, m, call):
    rec = Recorder(monkeypatch, m)
    made = ["zeros", "zeros"] if call is load else ["empty"]
    # a torch stream, a raw handle, the default stream by either of its handles
    for stream, on, launched in ((rec.Stream(77), 77, 77), (77, 77, 77), (0, 0, 0), (1, 0, 1)):
        call(m, rec, stream=stream)
        want = [x for name in made for x in ((name, on), ("kept for", "here"))]
        assert rec.steps == want + [("launch", launched)]
    call(m, rec, stream=None)
    assert rec.steps == [(name, "current") for name in made] + [("launch", "current")]


def test_given_tensors_are_not_filled(monkeypatch, m):
    rec = Recorder(monkeypatch, m)
    k, v = (torch.ones((3, 8, 128), dtype=torch.bfloat16) for _ in range(2))
    got = load(m, rec, k=k, v=v, stream=77)
    assert got[0] is k and got[1] is v
    assert rec.steps == [("launch", 77)] and bool((k == 1).all()) and bool((v == 1).all())
    got_k, got_v = load(m, rec, v=v, stream=77)
    assert got_v is v and rec.steps == [("zeros", 77), ("kept for", "here"), ("launch", 77)]
    assert not bool(got_k.any())
