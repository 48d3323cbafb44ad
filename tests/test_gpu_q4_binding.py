"""What the binding of the 4-bit calls refuses before anything is launched, and calls of size 0."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


def rows(n, heads, dtype=BF16, device="cuda"):
    return torch.zeros((n, heads, 128), dtype=dtype, device=device)


def i32(*x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


class Args(dict):
    """Valid arguments of every call; a test replaces one."""

    def __init__(self, pkv, **kw):
        super().__init__(
            q=rows(2, 16), k=rows(2, 8), v=rows(2, 8), slots=i32(0, 256), kc=pkv.q4_cache(4).zero_(),
            vc=pkv.q4_cache(4).zero_(), bt=i32([0, -1], [1, -1]), ctx=i32(1, 1),
            ws=pkv.decode_q4_workspace(2, 512), cu=i32(0, 1, 2), out=None, ko=None, vo=None, plan=None)
        self.update(kw)
        self.pkv = pkv

    def store(self):
        self.pkv.pkv_store_kvcache_q4(self["k"], self["v"], self["kc"], self["vc"], self["slots"])

    def load(self):
        return self.pkv.pkv_load_kvcache_q4(self["kc"], self["vc"], self["slots"], k=self["ko"], v=self["vo"])

    def decode(self):
        return self.pkv.pkv_decode_q4(self["q"], self["kc"], self["vc"], self["bt"], self["ctx"], 512, 0.1, self["ws"],
                                      out=self["out"])

    def step(self):
        return self.pkv.pkv_store_decode_q4(self["q"], self["k"], self["v"], self["slots"], self["kc"], self["vc"],
                                            self["bt"], self["ctx"], 512, 0.1, self["ws"], out=self["out"])

    def prefill(self):
        return self.pkv.pkv_prefill_varlen_q4(self["q"], self["cu"], self["cu"], 1, 1, 0.1, self["kc"], self["vc"],
                                              self["bt"], out=self["out"], plan=self["plan"])


CALLS = ["store", "load", "decode", "step", "prefill"]


def bad(pkv):
    """name -> (calls it belongs to, a wrong value)"""
    cache, ws = pkv.q4_cache(4), pkv.decode_q4_workspace(2, 512)
    wrong = []
    for name in ("kc", "vc"):
        for x in (cache.cpu(), cache.view(torch.int8), pkv.q4_cache(3), pkv.q4_cache(4, 4), cache[:, :, :8],
                  cache.reshape(4, 8, -1), pkv.q4_cache(8)[::2]):
            wrong.append((CALLS, name, x))
    for x in (rows(2, 16, torch.float16), rows(2, 16, device="cpu"), rows(2, 16)[:, :, :64], rows(2, 16).flatten(1),
              rows(2, 32)[:, ::2], rows(16, 2).transpose(0, 1)):
        wrong.append((["decode", "step", "prefill"], "q", x))
    for name in ("k", "v"):
        for x in (rows(2, 8, torch.float16), rows(2, 8, device="cpu"), rows(2, 4), rows(1, 8), rows(2, 16)[:, ::2]):
            wrong.append((["store", "step"], name, x))
    for x in (i32(0, 256).long(), i32(0, 256, device="cpu"), i32(0, 1, 256, 2)[::2], i32(0)):
        wrong.append((["store", "step"], "slots", x))
    for x in (i32([0, -1], [1, -1]).long(), i32([0, -1], [1, -1], device="cpu"), i32([0, -1]), i32(0, 1),
              i32([0, 1], [0, 1]).t()):
        wrong.append((["decode", "step", "prefill"], "bt", x))
    for x in (i32(1), i32(1, 1).float(), i32(1, 1, device="cpu")):
        wrong.append((["decode", "step"], "ctx", x))
    for x in (ws.cpu(), ws.view(torch.int32), ws[::2]):
        wrong.append((["decode", "step"], "ws", x))
    for x in (rows(2, 16, torch.float16), rows(1, 16), rows(2, 32)[:, ::2], rows(2, 16, device="cpu")):
        wrong.append((["decode", "step", "prefill"], "out", x))
    for name in ("ko", "vo"):
        for x in (rows(2, 8, torch.float16), rows(3, 8), rows(2, 16)[:, ::2]):
            wrong.append((["load"], name, x))
    wrong += [(["prefill"], "cu", i32(0, 1, 2).long()), (["prefill"], "cu", i32(0, 1, 2, device="cpu")),
              (["prefill"], "plan", i32(0, 1).long())]
    return wrong


def test_valid_calls(pkv):
    for call in CALLS:
        getattr(Args(pkv), call)()
    torch.cuda.synchronize()
    assert pkv.pkv_device_error() == 0


def test_refused_arguments(pkv):
    for calls, name, x in bad(pkv):
        for call in calls:
            with pytest.raises(ValueError):
                getattr(Args(pkv, **{name: x}), call)()
                pytest.fail(f"{call} took {name} {tuple(x.shape)} {x.dtype} {x.device} {x.stride()}")


def test_refused_by_the_library(pkv):
    short = Args(pkv, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    odd = Args(pkv, q=rows(2, 24))                            # three query heads to a kv head
    shifted = Args(pkv, q=torch.zeros(2 * 2048 + 1, dtype=BF16, device="cuda")[1:].view(2, 16, 128))
    for args, calls in ((short, ["decode", "step"]), (odd, ["decode", "step", "prefill"]),
                        (Args(pkv, q=rows(2, 8)), ["prefill"]), (shifted, ["decode", "step", "prefill"])):
        for call in calls:
            with pytest.raises(pkv.PkvError):
                getattr(args, call)()


def test_sizes_of_zero(pkv):
    none = Args(pkv, q=rows(0, 16), k=rows(0, 8), v=rows(0, 8), slots=i32(), ctx=i32(),
                bt=torch.zeros((0, 2), dtype=torch.int32, device="cuda"), cu=i32(0))
    none.store()
    k, v = none.load()
    assert k.shape == v.shape == (0, 8, 128)
    for call in ("decode", "step", "prefill"):
        assert getattr(none, call)().shape == (0, 16, 128)
    # rows that belong to no sequence, and sequences without rows
    out = torch.full((2, 16, 128), 3.0, dtype=BF16, device="cuda")
    Args(pkv, out=out, cu=i32(0, 0, 0)).prefill()
    assert bool((out == 3.0).all()) and pkv.pkv_device_error() == 0
