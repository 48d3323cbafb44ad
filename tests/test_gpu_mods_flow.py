"""The rotary positions, the attention calls with modified scores and the eviction as an engine uses them together:
prompts stored turned, attended to, decoded for some steps with their attention added up, cut down, decoded on."""
import pytest
import torch

import mods_reference as R

pytestmark = pytest.mark.gpu
D, BS = 128, 256


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_kvh_gb300 as m
    m.pkv_device_error(clear=True)
    return m


def _dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("in_place", [False, True])
def test_prompts_steps_eviction_steps(pkv, dtype, in_place):
    f16 = dtype == torch.float16
    rope_store = pkv.pkv_rope_store_kvcache_f16 if f16 else pkv.pkv_rope_store_kvcache
    prefill = pkv.pkv_prefill_varlen_mod_f16 if f16 else pkv.pkv_prefill_varlen_mod
    decode = pkv.pkv_decode_mod_f16 if f16 else pkv.pkv_decode_mod
    hq, hkv, cap, scale = 8, 2, 20.0, D ** -0.5
    lens, steps, budget, first, recent = [300, 45, 520], 5, 200, 2, 40
    eps = torch.finfo(dtype).eps / 2
    g = torch.Generator(device="cuda").manual_seed(11)
    freqs, magnitude = pkv.rope_frequencies(D, 1e6, "yarn", factor=4.0, original_max_position=4096)
    per = [-(-(n + 2 * steps) // BS) for n in lens]
    blocks = sum(per) + (0 if in_place else len(lens))
    kc, vc = (torch.zeros((blocks, BS, hkv, D), dtype=dtype, device="cuda") for _ in range(2))
    weights = pkv.attention_weights(blocks, hkv)
    order = torch.randperm(sum(per), generator=torch.Generator().manual_seed(3)).tolist()
    tables = [[order.pop() for _ in range(k)] for k in per]
    width = max(per)
    table = lambda t: _dev([x + [-1] * (width - len(x)) for x in t])  # noqa: E731

    def qkv(n):
        t = torch.randn((n, (hq + 2 * hkv) * D), generator=g, device="cuda").to(dtype)
        return (t[:, :hq * D].unflatten(1, (hq, D)), t[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D)),
                t[:, (hq + hkv) * D:].unflatten(1, (hkv, D)))

    slot = lambda t, i: t[i // BS] * BS + i % BS  # noqa: E731
    held = [([], []) for _ in lens]   # per sequence and head the rows that the cache should hold, in order, in 64 bits

    # ---- the prompts ----
    q, k, v = qkv(sum(lens))
    positions = torch.cat([torch.arange(n, device="cuda") for n in lens])
    slots = _dev([slot(t, i) for t, n in zip(tables, lens) for i in range(n)])
    qt = rope_store(q, k, v, positions, freqs, kc, vc, slots, magnitude=magnitude)
    ref_q = R.rope(q, positions.cpu(), freqs.cpu(), False, magnitude)
    ref_k = R.rope(k, positions.cpu(), freqs.cpu(), False, magnitude)
    assert bool(((qt.cpu().double() - ref_q).abs() <= R.rope_bound(q, ref_q, D // 2, False, magnitude)).all())
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    out = prefill(qt, _dev(cu), _dev(cu), max(lens), max(lens), scale, k_cache=kc, v_cache=vc, block_tables=table(tables),
                  softcap=cap)
    for b, n in enumerate(lens):
        kk, vv = R.cache_rows(kc, tables[b], n), R.cache_rows(vc, tables[b], n)
        assert bool(((kk.cpu().double() - ref_k[cu[b]:cu[b + 1]]).abs()
                     <= R.rope_bound(k, ref_k, D // 2, False, magnitude)[cu[b]:cu[b + 1]]).all())
        assert torch.equal(vv, v[cu[b]:cu[b + 1]])
        ref, p, bound, _ = R.attention_rows(qt[cu[b]:cu[b + 1]], kk, vv, 0, scale, softcap=cap)
        size = torch.einsum("hnt,thd->nhd", p, vv.double().abs().repeat_interleave(hq // hkv, 1))
        room = 2 * eps * ref.abs() + size * (eps + 2 * 6.9e-6 * cap + 2.0 ** -18) + bound + 2.0 ** -25
        assert bool(((out[cu[b]:cu[b + 1]].double() - ref).abs() <= room).all())
        held[b] = (kk, vv)

    # ---- steps: every head may hold tokens of its own after the eviction ----
    want_w = [torch.zeros((hkv, n), dtype=torch.float64, device="cuda") for n in lens]
    length = list(lens)          # tokens in the cache
    at = list(lens)              # the next token's position in the text
    ws = pkv.decode_mod_workspace(len(lens), width * BS, hq, hkv, weights=True)

    def step():
        q, k, v = qkv(len(lens))
        slots = _dev([slot(t, n) for t, n in zip(tables, length)])
        qt = rope_store(q, k, v, _dev(at, torch.int64), freqs, kc, vc, slots, magnitude=magnitude)
        for b in range(len(lens)):
            length[b] += 1
            at[b] += 1
        out = decode(qt, kc, vc, table(tables), _dev(length), width * BS, scale, ws, softcap=cap, weights=weights)
        for b, n in enumerate(length):
            new_k, new_v = R.cache_rows(kc, tables[b], n)[n - 1:], R.cache_rows(vc, tables[b], n)[n - 1:]
            held[b] = (torch.cat((held[b][0], new_k)), torch.cat((held[b][1], new_v)))
            ref, p, bound, _ = R.attention_rows(qt[b:b + 1], *held[b], n - 1, scale, softcap=cap)
            assert bool(((out[b:b + 1].double() - ref).abs() <= ref.abs() * eps + bound + 2.0 ** -25).all())
            want_w[b] = torch.cat((want_w[b], torch.zeros((hkv, 1), dtype=torch.float64, device="cuda")), 1)
            want_w[b] += p[:, 0].unflatten(0, (hkv, -1)).sum(1)

    for _ in range(steps):
        step()
    for b, n in enumerate(length):
        got = weights[_dev(tables[b], torch.long)].transpose(0, 1).flatten(1)[:, :n].double()
        # a probability of at most 1 in 32 bits, off by 2^-15 of it with its score's error, in each of the steps
        assert bool(((got - want_w[b]).abs() <= want_w[b] * 2.0 ** -15 + 2.0 ** -20).all())

    # ---- the cut: by the weights that the cache holds ----
    got_w = [weights[_dev(t, torch.long)].transpose(0, 1).flatten(1)[:, :n].cpu() for t, n in zip(tables, length)]
    new = None if in_place else [[sum(per) + b] for b in range(len(lens))]
    kept, lens_now = pkv.pkv_evict_kvcache(kc, vc, weights, table(tables), _dev(length), width * BS, budget, first=first,
                                           recent=recent, new_block_tables=None if in_place else _dev(new))
    assert lens_now.tolist() == [min(n, budget) for n in length]
    for b, n in enumerate(length):
        rows = [R.evict_choice(got_w[b][h].tolist(), first, recent, budget) for h in range(hkv)]
        assert kept[b, :, :len(rows[0])].tolist() == rows
        pick = _dev(rows, torch.long)                                  # [hkv, kept]
        held[b] = tuple(torch.stack([x[pick[h], h] for h in range(hkv)], 1) for x in held[b])
        want_w[b] = torch.gather(want_w[b], 1, pick)
        length[b] = min(n, budget)
        if not in_place:
            tables[b] = new[b]
    for b, n in enumerate(length):
        assert torch.equal(R.cache_rows(kc, tables[b], n), held[b][0])
        assert torch.equal(R.cache_rows(vc, tables[b], n), held[b][1])
    for _ in range(steps):
        step()
    for b, n in enumerate(length):
        got = weights[_dev(tables[b], torch.long)].transpose(0, 1).flatten(1)[:, :n].double()
        assert bool(((got - want_w[b]).abs() <= want_w[b] * 2.0 ** -15 + 2.0 ** -19).all())
    assert pkv.pkv_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_blocks_far_into_a_large_cache(pkv, dtype):
    """Blocks whose elements lie beyond 2^32 give what the same rows at the start of a small cache give, bit for bit."""
    f16 = dtype == torch.float16
    rope_store = pkv.pkv_rope_store_kvcache_f16 if f16 else pkv.pkv_rope_store_kvcache
    prefill = pkv.pkv_prefill_varlen_mod_f16 if f16 else pkv.pkv_prefill_varlen_mod
    decode = pkv.pkv_decode_mod_f16 if f16 else pkv.pkv_decode_mod
    hq, hkv, n, scale = 16, 8, 700, D ** -0.5
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn((n, h, D), generator=g, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    positions = torch.arange(n, device="cuda")
    freqs, _ = pkv.rope_frequencies(D)
    results = []
    for blocks, used in ((8, [3, 0, 7, 5]), (16500, [16499, 2, 16390, 16450])):
        kc, vc = (torch.empty((blocks, BS, hkv, D), dtype=dtype, device="cuda") for _ in range(2))
        weights = pkv.attention_weights(blocks, hkv)
        table = _dev([used[:3]])
        slots = _dev([used[i // BS] * BS + i % BS for i in range(n)])
        qt = rope_store(q, k, v, positions, freqs, kc, vc, slots)
        cu = _dev([0, n])
        out = prefill(qt, cu, cu, n, n, scale, k_cache=kc, v_cache=vc, block_tables=table, softcap=20.0, window=300)
        ws = pkv.decode_mod_workspace(1, n, hq, hkv, weights=True)
        step = decode(qt[-1:], kc, vc, table, _dev([n]), n, scale, ws, softcap=20.0, weights=weights)
        kept, _ = pkv.pkv_evict_kvcache(kc, vc, weights, table, _dev([n]), n, 200, first=2, recent=30,
                                        new_block_tables=_dev([used[3:]]))
        results.append((qt, out, step, kept, kc[used], vc[used][3, :200], weights[used][:3]))
        kc_kept, vc_kept = kc[used[3], :200], vc[used[3], :200]
        for h in range(hkv):
            at = slots[kept[0, h].long()].long()
            assert torch.equal(kc_kept[:, h], kc.flatten(0, 1)[at, h]) and torch.equal(vc_kept[:, h], vc.flatten(0, 1)[at, h])
    for name, a, b in zip(("q", "prefill", "decode", "kept"), *results):
        assert torch.equal(a, b), name
    a, b = results[0][4], results[1][4]
    assert torch.equal(a[:2], b[:2]) and torch.equal(a[2, :n - 2 * BS], b[2, :n - 2 * BS])
    assert torch.equal(a[3, :200], b[3, :200])
    assert torch.equal(results[0][5], results[1][5]) and torch.equal(results[0][6], results[1][6])
    assert pkv.pkv_device_error() == 0


def test_two_threads_on_their_own_streams(pkv):
    """Calls of two threads at once, each on a stream of its own, give what they give one after another."""
    import threading
    hq, hkv, scale = 12, 4, D ** -0.5
    lens = [[900, 33, 1400, 257], [2100, 5, 640]]
    freqs, _ = pkv.rope_frequencies(D)
    work = []
    for seed, ls in enumerate(lens):
        g = torch.Generator(device="cuda").manual_seed(seed)
        per = [-(-n // BS) for n in ls]
        ids = iter(range(sum(per)))
        table = [[next(ids) for _ in range(k)] + [-1] * (max(per) - k) for k in per]
        rows = lambda h: torch.randn((sum(ls), h, D), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        work.append(dict(q=rows(hq), k=rows(hkv), v=rows(hkv), blocks=sum(per), table=_dev(table), lens=_dev(ls),
                         most=max(ls), cu=_dev([0] + torch.tensor(ls).cumsum(0).tolist()),
                         positions=torch.cat([torch.arange(n, device="cuda") for n in ls]),
                         slots=_dev([t[i // BS] * BS + i % BS for t, n in zip(table, ls) for i in range(n)]),
                         ws=pkv.decode_mod_workspace(len(ls), max(ls), hq, hkv, weights=True)))

    def run(w):
        kc, vc = (torch.zeros((w["blocks"], BS, hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        weights = pkv.attention_weights(w["blocks"], hkv)
        qt = pkv.pkv_rope_store_kvcache(w["q"], w["k"], w["v"], w["positions"], freqs, kc, vc, w["slots"])
        out = pkv.pkv_prefill_varlen_mod(qt, w["cu"], w["cu"], w["most"], w["most"], scale, k_cache=kc, v_cache=vc,
                                         block_tables=w["table"], softcap=30.0, window=500)
        step = pkv.pkv_decode_mod(qt[w["cu"][1:].long() - 1], kc, vc, w["table"], w["lens"], w["most"], scale, w["ws"],
                                  softcap=30.0, weights=weights)
        kept, _ = pkv.pkv_evict_kvcache(kc, vc, weights, w["table"], w["lens"], w["most"], 300, first=4, recent=50)
        return [qt, out, step, kept, kc, vc]

    want = [run(w) for w in work]
    torch.cuda.synchronize()
    failures = []

    def thread(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = run(work[i])
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    failures.append(i)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures and pkv.pkv_device_error() == 0
