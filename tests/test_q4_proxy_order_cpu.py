"""The decode's stages are written by bulk copies and, where a step's new row is put in, by ordinary stores. The copy
that fills such a stage again is ordered after those stores only by a proxy fence of the threads that made them, before
they meet the thread that starts the copy. A missing one can't be made to show, so the source is looked at."""
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))


def test_stores_to_a_stage_are_fenced_before_the_warp_meets():
    path = os.path.join(HERE, "..", "paged_kv_cache_kvh_gb300", "csrc", "q4_decode.cu")
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = text[text.index("q4_decode_kernel(const Q4DecodeParams p) {"):]
    stores = [m.start() for m in re.finditer(r"\bsts32\(", body)]
    assert len(stores) == 4                                    # codes and parameters, of K and of V
    for at in stores:
        rest = body[at:]
        assert 0 <= rest.find("fence_proxy_async_smem();") < rest.find("__syncwarp();")
