"""The package imports on a torch without the private allocation call that its newer entry points use where it is there."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
{remove}
import paged_kv_cache_kvh_gb300 as pkv
assert pkv._empty_cuda is pkv._empty_on_cuda
seen = []
torch.empty_strided = lambda shape, strides, **kw: seen.append((shape, strides, kw)) or "made"
assert pkv._empty_cuda((2, 3), (3, 1), torch.int32) == "made"
assert seen == [((2, 3), (3, 1), dict(dtype=torch.int32, device="cuda"))]
"""


@pytest.mark.parametrize("remove", ["if hasattr(torch._C._dynamo.guards, '_empty_strided_cuda'): "
                                    "del torch._C._dynamo.guards._empty_strided_cuda",
                                    "del torch._C._dynamo.guards", "del torch._C._dynamo"])
def test_without_the_private_allocation_call(remove):
    pytest.importorskip("torch")
    done = subprocess.run([sys.executable, "-c", SCRIPT.format(remove=remove)], cwd=ROOT, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr[-2000:]
