"""A worker of the decode with modified scores whose wait runs out leaves without its partial results. The joining kernel
must not take sequence and range numbers from what then stands in the workspace, which needs no initialisation. A wait
cannot be made to run out there, so the source is looked at, and its rule for what is followed is tried."""
import os
import random
import re

HERE = os.path.dirname(os.path.abspath(__file__))


def _source():
    with open(os.path.join(HERE, "..", "paged_kv_cache_kvh_gb300", "csrc", "decode_mod.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_a_worker_says_that_nothing_goes_on_before_it_waits():
    text = _source()
    body = text[text.index("decode_mod_kernel(const __grid_constant__"):text.index("__device__ __forceinline__ void join(")]
    loop = body[body.index("for (int stream = first_stream;"):]
    assert 0 <= loop.find("if (tells) p.info[range].seq = -1;") < loop.find("mbar_wait(")
    assert "const bool tells = !by_cta && stream == 0 && lane == 0;" in loop
    # whoever writes what goes on is the one who has said so, later in the same program
    assert loop.find("if (tells) {") > loop.find("mbar_wait(")


def test_only_entries_that_fit_are_followed():
    text = _source()
    kernel = text[text.index("decode_mod_merge_kernel(const DecodeModParams p) {"):]
    read, check = kernel.index("p.info + first + warp"), kernel.index("if (!fits(p, first + warp, info.x, info.y, info.z)) info.x = -1;")
    assert read < check < kernel.index("join(") and check < kernel.index("s_info[warp][0] = info.x;")
    rule = re.search(r"bool fits\([^)]*\) \{\s*return (.*?);", text, re.S).group(1)
    rule = rule.replace("&&", " and ").replace("p.", "p_").replace("\n", " ")
    rng = random.Random(1)
    edges = [-2 ** 31, -1, 0, 1, 2, 15, 16, 17, 151, 152, 2 ** 24, 2 ** 31 - 1]
    for _ in range(20000):
        seqs, used = rng.choice([1, 14, 65535]), rng.choice([1, 2, 19, 152, 1216])
        r = rng.randrange(used)
        seq, last, place = (rng.choice(edges + [rng.randrange(-2 ** 31, 2 ** 31), seqs - 1, seqs, r, used - 1, used]) for _ in range(3))
        got = eval(rule, dict(p_num_seqs=seqs, p_used_ranges=used, range=r, seq=seq, last=last, place=place))
        assert got == (0 <= seq < seqs and r <= last <= used - 1 and place in (0, 1))
