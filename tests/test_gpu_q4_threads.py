"""The first 4-bit calls of a process made by several host threads at once."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

PROGRAM = """
import sys, threading
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import paged_kv_cache_kvh_gb300 as pkv
from test_gpu_q4_prefill import Prefill
BF16, F16 = torch.bfloat16, torch.float16
cases = [Prefill(pkv, [200, 33], [900, 33], hq, 4, t, seed=91 + i)
         for i, (hq, t) in enumerate([(8, BF16), (8, F16), (16, BF16), (16, F16)] * 2)]
first = threading.Barrier(len(cases))
got, failed = {{}}, []

def work(i):
    try:
        c, s = cases[i], torch.cuda.Stream()
        q = c.q[:2]
        ws = c.pkv.decode_q4_workspace(2, c.max_ctx, c.hq, c.hkv)
        torch.cuda.synchronize()
        first.wait(60)
        with torch.cuda.stream(s):
            c.fill()
            out = c.prefill()
            dec = c.f("pkv_decode_q4")(q, c.kc, c.vc, c.tables, c.ctx, c.max_ctx, c.scale, ws)
        s.synchronize()
        got[i] = out, dec, ws
    except BaseException as e:
        failed.append((i, repr(e)))

threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
for t in threads: t.start()
for t in threads: t.join(120)
assert not failed and len(got) == len(cases), failed
for i, c in enumerate(cases):
    out, dec, ws = got[i]
    c.check(out)
    assert torch.equal(out, c.prefill())
    again = c.f("pkv_decode_q4")(c.q[:2], c.kc, c.vc, c.tables, c.ctx, c.max_ctx, c.scale, ws)
    assert torch.equal(dec, again)
assert pkv.pkv_device_error() == 0
print("done")
"""


def test_first_calls_of_several_threads():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    code = PROGRAM.format(root=os.path.dirname(HERE), tests=HERE)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), r.stdout + r.stderr
