"""Cases of what comes before, inside and after attention over the paged cache.

Kinds of cases:
  "rotate"        queries and keys [N, heads, 128] turned by their positions
  "rotate_store"  the same, with the turned keys and the values written to their slots
  "decode"        one query token for each sequence over the paged cache, with scores
                  that may be capped, get a bias by distance and see a part of the
                  keys; with "weights" each key's attention is added up beside it
  "prefill"       variable-length attention of new tokens, keys contiguous or paged,
                  with the same scores and a visible range of keys for each row
  "evict"         for each sequence and kv head the cached tokens with the largest
                  added-up attention (and the first and the newest ones) copied to
                  new blocks

Rotation: pair i of a head turns by position * freqs[i] / 2^64 of a full turn; the
frequencies are 64-bit fixed-point numbers, so the product's low 64 bits are exact.
Scores: s = scale * q.k, then cap * tanh(s / cap), then - slope[head] * |p - t| for a
query at position p and a key at position t. A key is visible where start <= t,
t <= p or t < prefix, t < length, and p - t < window.
"""
import math
import random

import torch

own = False

D, BS = 128, 256
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
THETA = 1e6


# ---- cases ----------------------------------------------------------------------------


def listed():
    return [
        # one step of a few users: a call's latency
        dict(name="rotate_step", kind="rotate", dtype="bf16", hq=16, hkv=8, rot=128, layout="half", scaling="none",
             seqs=5, lo=1, hi=1, lens_seed=1, max_pos=4096),
        # the rows of one call of prompts, just below 16384 tokens
        dict(name="rotate_prompts", kind="rotate", dtype="fp16", hq=16, hkv=8, rot=64, layout="interleaved",
             scaling="linear", factor=4.0, seqs=29, lo=100, hi=1024, lens_seed=7, max_pos=8192),
        # the new rows of a decode step of 256 sequences: one token to a block
        dict(name="rotate_store_step", kind="rotate_store", dtype="bf16", hq=16, hkv=8, rot=128, layout="half",
             scaling="none", seqs=256, lo=1, hi=1, lens_seed=4, max_pos=4096),
        # a call of prompts far into long contexts, frequencies stretched by parts
        dict(name="rotate_store_prompts", kind="rotate_store", dtype="bf16", hq=16, hkv=8, rot=128, layout="half",
             scaling="yarn", factor=4.0, original=32768, seqs=29, lo=100, hi=1024, lens_seed=7, max_pos=131072),
        # a small step with ragged contexts from one token on, a bias by distance, a window, padding rows
        dict(name="decode_small_biased", kind="decode", dtype="fp16", hq=12, hkv=12, seqs=14, lo=1, hi=2500, lens_seed=3,
             pad=2, max_context=4096, cap=0.0, bias=True, window=1000, docs=0, weights=False, sharp=2.0),
        # a serving batch whose scores are capped and whose attention is added up for a later eviction
        dict(name="decode_batch_weights", kind="decode", dtype="bf16", hq=16, hkv=8, seqs=256, lo=512, hi=4096,
             lens_seed=2, pad=0, max_context=4096, cap=50.0, bias=False, window=0, docs=0, weights=True, sharp=3.0),
        # one user with a long context: few rows, a long axis to split; 4 query heads to a kv head, capped
        dict(name="decode_one_long_capped", kind="decode", dtype="bf16", hq=32, hkv=8, lens="40007", pad=0,
             max_context=40960, cap=30.0, bias=False, window=0, docs=0, weights=False, sharp=4.0),
        # a call of prompts, capped, each row over the last 300 keys
        dict(name="prefill_prompts_window", kind="prefill", dtype="bf16", hq=16, hkv=8, seqs=29, lo=100, hi=1024,
             lens_seed=7, cached=0, paged=False, cap=50.0, bias=False, window=300, docs=0, prefix=0, sharp=3.0),
        # documents of about 700 tokens packed into rows, behind cached tokens, with a prefix that all rows see
        dict(name="prefill_documents", kind="prefill", dtype="fp16", hq=16, hkv=8, seqs=6, lo=1800, hi=4096, lens_seed=9,
             cached=300, paged=True, cap=0.0, bias=True, window=0, docs=700, prefix=400, sharp=2.0),
        # a chunk of a long prompt, capped: 5000 new tokens behind 7001 cached ones
        dict(name="prefill_chunk_capped", kind="prefill", dtype="bf16", hq=16, hkv=8, lens="5000", cached=7001,
             paged=True, cap=50.0, bias=False, window=0, docs=0, prefix=0, sharp=3.0),
        # one long context cut to a quarter
        dict(name="evict_one_long", kind="evict", dtype="bf16", hkv=8, lens="40007", max_context=40960, budget=10000,
             first=4, recent=512),
        # a batch cut to at most 1500 tokens each
        dict(name="evict_batch", kind="evict", dtype="fp16", hkv=8, seqs=96, lo=512, hi=4096, lens_seed=2,
             max_context=4096, budget=1500, first=16, recent=256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(16, 8), (16, 8), (32, 8), (12, 12), (8, 2), (4, 1), (9, 3), (20, 2)]


def draw(rng):
    kind = rng.choice(["rotate", "rotate_store", "decode", "decode", "prefill", "prefill", "evict"])
    dtype = rng.choice(["bf16", "fp16"])
    hq, hkv = rng.choice(HEADS)
    seed = rng.randrange(1 << 30)
    if kind in ("rotate", "rotate_store"):
        seqs = _log_int(rng, 1, 256)
        hi = max(1, min(_log_int(rng, 1, 4096), 14000 * 24 // (hq + hkv) // seqs))
        scaling = rng.choice(["none", "linear", "ntk", "bands", "yarn"])
        return dict(kind=kind, dtype=dtype, hq=hq, hkv=hkv, rot=rng.choice([128, 128, 64, 32, 96, 6]),
                    layout=rng.choice(["half", "interleaved"]), scaling=scaling, factor=rng.choice([2.0, 4.0, 8.5]),
                    original=rng.choice([4096, 8192, 32768]), seqs=seqs, lo=max(1, hi // 3), hi=hi, lens_seed=seed,
                    max_pos=_log_int(rng, 4096, 2000000))
    cap, bias = rng.choice([0.0, 0.0, 20.0, 30.0, 50.0]), rng.choice([False, False, True])
    sharp = rng.choice([1.0, 2.0, 4.0])
    if kind == "decode":
        # at most 590,000 cached tokens of 8 kv heads, the size of the largest listed batch
        seqs = _log_int(rng, 1, 512)
        hi = max(1, min(_log_int(rng, 8, 40000), 590000 * 8 // hkv // seqs, 590000 // seqs))
        return dict(kind=kind, dtype=dtype, hq=hq, hkv=hkv, seqs=seqs, lo=max(1, hi // rng.randint(1, 8)), hi=hi,
                    lens_seed=seed, pad=rng.choice([0, 0, 1, 9]), max_context=hi + rng.choice([0, 1, 1000]), cap=cap,
                    bias=bias, window=rng.choice([0, 0, 1, _log_int(rng, 16, 4096)]),
                    docs=rng.choice([0, 0, _log_int(rng, 50, 5000)]), weights=rng.choice([False, True]), sharp=sharp)
    if kind == "evict":
        seqs = _log_int(rng, 1, 128)
        hi = max(2, min(_log_int(rng, 2, 40000), 230000 // seqs))
        budget = max(1, min(int(hi * rng.uniform(0.1, 1.1)), 12000 if seqs > 8 else 40000))
        first = min(budget, rng.choice([0, 1, 4, 100]))
        return dict(kind=kind, dtype=dtype, hkv=rng.choice([8, 8, 2, 5, 1]), seqs=seqs, lo=max(1, hi // 5), hi=hi,
                    lens_seed=seed, max_context=hi + rng.choice([0, 1, 300]), budget=budget, first=first,
                    recent=min(budget - first, rng.choice([0, 1, 32, 333])))
    if hq > 16:
        hq, hkv = 16, 8
    seqs = _log_int(rng, 1, 64)
    hi = max(1, min(_log_int(rng, 1, 4000), 10000 // seqs))
    return dict(kind=kind, dtype=dtype, hq=hq, hkv=hkv, seqs=seqs, lo=max(1, hi // 4), hi=hi, lens_seed=seed,
                cached=rng.choice([0, 1, 300, 1024, 2500]) if seqs <= 16 else rng.choice([0, 0, 513]),
                paged=rng.choice([True, False]), cap=cap, bias=bias, window=rng.choice([0, 0, 0, _log_int(rng, 1, 3000)]),
                docs=rng.choice([0, 0, _log_int(rng, 20, 2000)]), prefix=rng.choice([0, 0, 1, 200, 1500]), sharp=sharp)


def _lens(case):
    """The sequences' new or cached lengths, the same for every seed."""
    if "lens" in case:
        return [int(x) for x in case["lens"].split(",")]
    rng = random.Random(case["lens_seed"])
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


def _doc_starts(case, lengths):
    """For each sequence the start of each position's document (a list of positions), or None without documents."""
    mean = case.get("docs", 0)
    if not mean:
        return None
    rng = random.Random(case.get("lens_seed", 0) + 1)
    found = []
    for n in lengths:
        starts, at = [], 0
        while at < n:
            size = min(n - at, max(1, int(rng.expovariate(1.0 / mean))))
            starts += [at] * size
            at += size
        found.append(starts)
    return found


def _inverse_frequencies(case):
    """Radians per position of each pair, and the factor of the turned values."""
    r, factor, base = case["rot"], case.get("factor", 1.0), THETA
    scaling, orig = case["scaling"], case.get("original", 4096)
    if scaling == "ntk" and r > 2:
        base *= factor ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "bands":  # wavelengths beyond original / 1 stretched, those below original / 4 kept, a ramp between
        keep = [min(1.0, max(0.0, (orig * x / (2 * math.pi) - 1.0) / 3.0)) for x in f]
        return [x / factor * (1 - g) + x * g for x, g in zip(f, keep)], 1.0
    if scaling == "yarn":  # pairs that turn 32 times over the original length kept, those below once stretched
        def pair(turns):
            return r * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(0, math.floor(pair(32.0))), min(r - 1, math.ceil(pair(1.0)))
        ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(r // 2)]
        return [x / factor * g + x * (1 - g) for x, g in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ---- states -----------------------------------------------------------------------------


def _tables(lens, rng, spare=16):
    """Block tables (host lists) of sequences of these lengths, and the number of blocks with some spare ones."""
    order = list(range(sum(-(-n // BS) for n in lens) + spare))
    rng.shuffle(order)
    tables, at = [], 0
    for n in lens:
        tables.append(order[at:at + -(-n // BS)])
        at += -(-n // BS)
    return tables, len(order)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    lens, dtype, hkv, kind = _lens(case), DTYPES[case["dtype"]], case["hkv"], case["kind"]
    hq = case.get("hq", hkv)
    st = dict(case=case, dtype=dtype, scale=1.0 / math.sqrt(D))

    def dev(a, dt=torch.int32):
        return torch.tensor(a, dtype=dt, device="cuda")

    def normal(shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    def pool(blocks):
        return normal((blocks, BS, hkv, D)), normal((blocks, BS, hkv, D))

    def qkv(n, scale=1.0):
        # views of one fused projection, as attention layers get them
        t = normal((n, (hq + 2 * hkv) * D))
        q = t[:, :hq * D].unflatten(1, (hq, D))
        q.mul_(scale)
        return (q, t[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D)), t[:, (hq + hkv) * D:].unflatten(1, (hkv, D)))

    def padded(tables, width):
        return dev([t + [-1] * (width - len(t)) for t in tables])

    if kind in ("rotate", "rotate_store"):
        f, st["magnitude"] = _inverse_frequencies(case)
        st["freqs"] = dev([int(x / (2 * math.pi) * 2.0 ** 64) for x in f], torch.int64)
        st["q"], st["k"], st["v"] = qkv(sum(lens))
        first = [rng.randint(0, case["max_pos"] - n) if case["max_pos"] > n else 0 for n in lens]
        st["positions"] = torch.cat([torch.arange(a, a + n, device="cuda") for a, n in zip(first, lens)])
        if kind == "rotate_store":
            tables, blocks = _tables(lens, rng)
            st["slots"] = dev([t[i // BS] * BS + i % BS for t, n in zip(tables, lens) for i in range(n)])
            st["k_cache"], st["v_cache"] = pool(blocks)
        return st
    slopes = [2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]
    if kind == "decode":
        pad, longest = case["pad"], max(case["max_context"], max(lens))
        tables, blocks = _tables(lens, rng)
        st["k_cache"], st["v_cache"] = pool(blocks)
        st["block_tables"] = padded(tables + [[]] * pad, -(-longest // BS))
        st["context_lens"] = dev(lens + [0] * pad)
        st["max_context"] = longest
        st["q"] = qkv(len(lens) + pad, case["sharp"])[0]
        docs = _doc_starts(case, lens)
        st["key_starts"] = None if docs is None else dev([d[-1] for d in docs] + [0] * pad)
        st["weights"] = (torch.rand((blocks, hkv, BS), generator=gen, device="cuda") if case["weights"] else None)
        st["live"], st["width"] = len(lens), -(-max(lens) // BS)
    elif kind == "prefill":
        cached = case["cached"]
        totals = [n + cached for n in lens]
        cu_q, cu_k = [0], [0]
        for n in lens:
            cu_q.append(cu_q[-1] + n)
            cu_k.append(cu_k[-1] + n + cached)
        st.update(cu_q=dev(cu_q), cu_k=dev(cu_k), max_q=max(lens), max_k=max(totals))
        st["q"], new_k, new_v = qkv(cu_q[-1], case["sharp"])
        if case["paged"]:
            tables, blocks = _tables(totals, rng)
            st["k_cache"], st["v_cache"] = pool(blocks)
            st["block_tables"] = padded(tables, -(-max(totals) // BS))
        elif cached:
            st["k"], st["v"] = normal((cu_k[-1], hkv, D)), normal((cu_k[-1], hkv, D))
        else:
            st["k"], st["v"] = new_k, new_v
        docs = _doc_starts(case, totals)
        st["key_starts"] = None if docs is None else dev([x for d in docs for x in d[cached:]])
        st["prefix_lens"] = dev([case["prefix"]] * len(lens)) if case["prefix"] else None
    else:
        budget = case["budget"]
        tables, blocks = _tables(lens, rng)
        more, new = _tables([min(n, budget) for n in lens], rng, 0)
        st["k_cache"], st["v_cache"] = pool(blocks + new)
        w = torch.randn((blocks + new, hkv, BS), generator=gen, device="cuda")
        st["weights"] = torch.where(w < -0.8, torch.zeros_like(w), torch.exp(2.5 * w))  # heavy-tailed, some never seen
        longest = max(case["max_context"], max(lens))
        st["block_tables"] = padded(tables, -(-longest // BS))
        st["new_tables"] = padded([[b + blocks for b in t] for t in more], -(-budget // BS))
        st["context_lens"] = dev(lens)
        st.update(max_context=longest, first_new=blocks, width=-(-max(lens) // BS))
        return st
    st["slopes"] = dev(slopes, torch.float32) if case["bias"] else None
    return st


# ---- one pass ---------------------------------------------------------------------------


def run(st):
    case, kind = st["case"], st["case"]["kind"]
    if own:
        import paged_kv_cache_kvh_gb300 as pkv
        f16 = st["dtype"] == torch.float16
        if kind == "rotate":
            rope = pkv.pkv_rope_f16 if f16 else pkv.pkv_rope
            return rope(st["q"], st["k"], st["positions"], st["freqs"], magnitude=st["magnitude"],
                        interleaved=case["layout"] == "interleaved")
        if kind == "rotate_store":
            rope = pkv.pkv_rope_store_kvcache_f16 if f16 else pkv.pkv_rope_store_kvcache
            q = rope(st["q"], st["k"], st["v"], st["positions"], st["freqs"], st["k_cache"], st["v_cache"], st["slots"],
                     magnitude=st["magnitude"], interleaved=case["layout"] == "interleaved")
            return q, st["k_cache"], st["v_cache"]
        if kind == "decode":
            if "workspace" not in st:  # kept by the engine for all its steps
                st["workspace"] = pkv.decode_mod_workspace(st["q"].shape[0], st["max_context"], case["hq"], case["hkv"],
                                                           weights=case["weights"])
            decode = pkv.pkv_decode_mod_f16 if f16 else pkv.pkv_decode_mod
            out = decode(st["q"], st["k_cache"], st["v_cache"], st["block_tables"], st["context_lens"],
                         st["max_context"], st["scale"], st["workspace"], softcap=case["cap"], slopes=st["slopes"],
                         window=case["window"], key_starts=st["key_starts"], weights=st["weights"])
            return (out, st["weights"]) if case["weights"] else out
        if kind == "prefill":
            prefill = pkv.pkv_prefill_varlen_mod_f16 if f16 else pkv.pkv_prefill_varlen_mod
            keys = ({"k_cache": st["k_cache"], "v_cache": st["v_cache"], "block_tables": st["block_tables"]}
                    if case["paged"] else {"k": st["k"], "v": st["v"]})
            return prefill(st["q"], st["cu_q"], st["cu_k"], st["max_q"], st["max_k"], st["scale"], **keys,
                           softcap=case["cap"], slopes=st["slopes"], window=case["window"], key_starts=st["key_starts"],
                           prefix_lens=st["prefix_lens"])
        kept, lens = pkv.pkv_evict_kvcache(st["k_cache"], st["v_cache"], st["weights"], st["block_tables"],
                                           st["context_lens"], st["max_context"], case["budget"], first=case["first"],
                                           recent=case["recent"], new_block_tables=st["new_tables"])
    else:
        if kind == "rotate":
            return _rotate(st, st["q"]), _rotate(st, st["k"])
        if kind == "rotate_store":
            at = st["slots"].long()
            st["k_cache"].flatten(0, 1)[at] = _rotate(st, st["k"])
            st["v_cache"].flatten(0, 1)[at] = st["v"]
            return _rotate(st, st["q"]), st["k_cache"], st["v_cache"]
        if kind == "decode":
            return _decode(st)
        if kind == "prefill":
            return _prefill(st)
        kept, lens = _evict(st)
    return kept, lens, st["k_cache"][st["first_new"]:], st["v_cache"][st["first_new"]:], st["weights"][st["first_new"]:]


def _rotate(st, x):
    """The products' low 64 bits are the turn's fraction; angles, cosines and sines in 64 bits, the turning in 32."""
    rot = st["case"]["rot"]
    angle = (st["positions"][:, None] * st["freqs"]).double() * (2 * math.pi / 2.0 ** 64)
    cos = (angle.cos() * st["magnitude"]).float()[:, None]
    sin = (angle.sin() * st["magnitude"]).float()[:, None]
    y = x[..., :rot].float()
    if st["case"]["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned.to(x.dtype), x[..., rot:]), -1)


def _softmax_rows(s, seen):
    """Probabilities of the seen keys; rows that see none get zeros."""
    s = s.masked_fill_(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True)
    e = s.sub_(torch.where(top == float("-inf"), torch.zeros_like(top), top)).exp_()
    total = e.sum(-1, keepdim=True)
    return e.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _scores(st, s, distance):
    """Raw scores [B, hkv, group, rows, keys] in 32 bits, distance [B, rows, keys]."""
    case = st["case"]
    s = s.mul_(st["scale"])
    if case["cap"]:
        s = s.div_(case["cap"]).tanh_().mul_(case["cap"])
    if st["slopes"] is not None:
        s = s.sub_(st["slopes"].unflatten(0, (case["hkv"], -1))[:, :, None, None] * distance[:, None, None].abs())
    return s


def _decode(st):
    """One query for each sequence; rows that see no key give zeros."""
    case, live, hkv = st["case"], st["live"], st["case"]["hkv"]
    tables = st["block_tables"][:live, :st["width"]].long().clamp(min=0)
    q = st["q"][:live].float().unflatten(1, (hkv, -1))
    n = st["context_lens"][:live].long()
    t = torch.arange(tables.shape[1] * BS, device=q.device)
    distance = n[:, None] - 1 - t
    seen = distance >= 0
    if st["key_starts"] is not None:
        seen = seen & (t >= st["key_starts"][:live, None])
    if case["window"]:
        seen = seen & (distance < case["window"])
    s = torch.einsum("bhgd,bthd->bhgt", q, st["k_cache"][tables].flatten(1, 2).float())
    p = _softmax_rows(_scores(st, s[:, :, :, None], distance[:, None].float())[:, :, :, 0], seen[:, None, None])
    out = torch.zeros(st["q"].shape, dtype=st["dtype"], device=q.device)
    out[:live] = torch.einsum("bhgt,bthd->bhgd", p, st["v_cache"][tables].flatten(1, 2).float()).flatten(1, 2)
    if not case["weights"]:
        return out
    # a token's sum starts from 0 in the step that stores it
    b, i = torch.nonzero(seen | (distance == 0), as_tuple=True)
    block, place = tables[b, i // BS], i % BS
    before = st["weights"][block, :, place]
    before = torch.where((distance[b, i] == 0)[:, None], torch.zeros_like(before), before)
    st["weights"][block, :, place] = before + p.sum(2)[b, :, i]
    return out, st["weights"]


def _prefill(st):
    """Sequences padded to the longest; query row i of a sequence sits at position Lk - Lq + i."""
    case, hkv = st["case"], st["case"]["hkv"]
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    lq, lk = cu_q.diff(), cu_k.diff()
    rows = torch.arange(st["q"].shape[0], device=cu_q.device)
    seq = torch.searchsorted(cu_q, rows, right=True) - 1
    i, t = torch.arange(st["max_q"], device=cu_q.device), torch.arange(st["max_k"], device=cu_q.device)
    take = (cu_q[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    if case["paged"]:
        at = st["block_tables"].long().clamp(min=0)[:, t // BS] * BS + t % BS
        k, v = st["k_cache"].flatten(0, 1)[at], st["v_cache"].flatten(0, 1)[at]
    else:
        at = (cu_k[:-1, None] + t).clamp(max=st["k"].shape[0] - 1)
        k, v = st["k"][at], st["v"][at]
    distance = (lk - lq)[:, None, None] + i[:, None] - t                      # [B, Lq, T]
    seen = distance >= 0
    if st["prefix_lens"] is not None:
        seen = seen | (t < st["prefix_lens"][:, None, None])
    seen = seen & (t < lk[:, None, None])
    if st["key_starts"] is not None:
        seen = seen & (t >= st["key_starts"][take][..., None])
    if case["window"]:
        seen = seen & (distance < case["window"])
    q = st["q"][take].float().unflatten(2, (hkv, -1))                         # [B, Lq, hkv, g, d]
    s = _scores(st, torch.einsum("bihgd,bthd->bhgit", q, k.float()), distance.float())
    p = _softmax_rows(s, seen[:, None, None])
    o = torch.einsum("bhgit,bthd->bihgd", p, v.float()).flatten(2, 3)
    return o[seq, rows - cu_q[seq]].to(st["dtype"])


def _evict(st):
    """Kept positions in rising order (-1 behind them) and the new lengths; rows and sums go to the new blocks."""
    case, hkv, budget = st["case"], st["case"]["hkv"], st["case"]["budget"]
    tables, new = st["block_tables"][:, :st["width"]].long().clamp(min=0), st["new_tables"].long().clamp(min=0)
    n = st["context_lens"].long()[:, None, None]
    w = st["weights"][tables].transpose(1, 2).flatten(2)                      # [B, hkv, T]
    t = torch.arange(w.shape[-1], device=w.device)
    safe = (t < case["first"]) | (t >= n - case["recent"])
    order = torch.where(t < n, torch.where(safe, float("inf"), w), float("-inf"))
    rank = torch.sort(order, dim=-1, descending=True, stable=True).indices[..., :budget]
    some = torch.arange(rank.shape[-1], device=w.device) < n
    kept = torch.sort(torch.where(some, rank, t.shape[0]), dim=-1).values
    b, h, j = torch.nonzero(kept < t.shape[0], as_tuple=True)
    source = kept[b, h, j]
    fb, fi, tb, ti = tables[b, source // BS], source % BS, new[b, j // BS], j % BS
    st["k_cache"][tb, ti, h] = st["k_cache"][fb, fi, h]
    st["v_cache"][tb, ti, h] = st["v_cache"][fb, fi, h]
    st["weights"][tb, h, ti] = st["weights"][fb, h, fi]
    out = torch.full((n.shape[0], hkv, budget), -1, dtype=torch.int32, device=w.device)
    out[b, h, j] = source.int()
    return out, st["context_lens"].clamp(max=budget)


# ---- what a pass cannot do without --------------------------------------------------------


def work(case):
    lens, hkv, kind = _lens(case), case["hkv"], case["kind"]
    hq, row = case.get("hq", hkv), 2 * D
    if kind in ("rotate", "rotate_store"):
        n = sum(lens)
        moved = 2 * n * (hq + hkv) * row + 8 * n
        return {"bytes": moved + (2 * n * hkv * row + 4 * n if kind == "rotate_store" else 0), "flops": 0}
    if kind == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": hkv * (4 * sum(lens) + kept * (4 * row + 8) + kept * 4), "flops": 0}
    if kind == "decode":
        docs = _doc_starts(case, lens)
        seen = [n - max(docs[i][-1] if docs else 0, n - case["window"] if case["window"] else 0)
                for i, n in enumerate(lens)]
        moved = sum(seen) * hkv * (2 * row + (8 if case["weights"] else 0)) + 2 * (len(lens) + case["pad"]) * hq * row
        return {"bytes": moved + 4 * sum(-(-n // BS) for n in lens), "flops": 4 * D * hq * sum(seen)}
    cached, prefix, window, pairs, keys = case["cached"], case["prefix"], case["window"], 0, 0
    docs = _doc_starts(case, [n + cached for n in lens])
    for i, n in enumerate(lens):
        total, least = n + cached, n + cached
        for p in range(cached, total):
            lo = max(docs[i][p] if docs else 0, p - window + 1 if window else 0)
            pairs += max(0, min(total, max(p + 1, prefix)) - lo)
            least = min(least, lo)
        keys += total - least
    return {"bytes": keys * hkv * 2 * row + 2 * sum(lens) * hq * row, "flops": 4 * D * hq * pairs}


# ---- the definition in 64 bits --------------------------------------------------------------


def _exact_turned(x, positions, case):
    """Each pair as a complex number times magnitude * e^(i position f), f in radians."""
    f, magnitude = _inverse_frequencies(case)
    r = case["rot"]
    turn = torch.polar(torch.full((len(positions), r // 2), magnitude, dtype=torch.float64, device="cuda"),
                       positions.double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda"))
    out = x.double().clone()
    first, second = ((slice(0, r // 2), slice(r // 2, r)) if case["layout"] == "half"
                     else (slice(0, r, 2), slice(1, r, 2)))
    z = torch.complex(out[..., first], out[..., second]) * turn[:, None]
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rows(st, q, k, v, first, starts, prefix):
    """Rows [n, hq, 128] at positions first, first + 1, ... over keys [T, hkv, 128]: outputs and probabilities [hq, n, T]."""
    case = st["case"]
    g = case["hq"] // case["hkv"]
    s = torch.einsum("nhd,thd->hnt", q.double(), k.double().repeat_interleave(g, 1)) / math.sqrt(D)
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    p = first + torch.arange(q.shape[0], device="cuda")[:, None]
    t = torch.arange(k.shape[0], device="cuda")
    if case["bias"]:
        slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / case["hq"]) for h in range(case["hq"])], device="cuda")
        s = s - slopes.double()[:, None, None] * (p - t).abs().double()
    hidden = ((t > p) & (t >= prefix)) | (t < starts[:, None])
    if case["window"]:
        hidden = hidden | (p - t >= case["window"])
    e = torch.softmax(s.masked_fill(hidden, float("-inf")), -1).nan_to_num(0.0)
    return torch.einsum("hnt,thd->nhd", e, v.double().repeat_interleave(g, 1)), e


def exact(case, seed):
    st = prepare(case, seed)
    lens, kind = _lens(case), case["kind"]
    if kind == "evict":
        return None  # whole numbers and copies
    if kind == "rotate":
        return tuple(_exact_turned(st[x], st["positions"], case) for x in "qk")
    if kind == "rotate_store":
        q, k = (_exact_turned(st[x], st["positions"], case) for x in "qk")
        caches = st["k_cache"].double(), st["v_cache"].double()
        for cache, rows in zip(caches, (k, st["v"].double())):
            cache.view(-1, *rows.shape[1:])[st["slots"].long()] = rows
        return (q, *caches)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    if kind == "decode":
        weights = st["weights"].double() if case["weights"] else None
        for b, n in enumerate(lens):
            blocks = st["block_tables"][b, :-(-n // BS)].long()
            k, v = (c[blocks].flatten(0, 1)[:n] for c in (st["k_cache"], st["v_cache"]))
            start = none if st["key_starts"] is None else st["key_starts"][b:b + 1].long()
            out[b:b + 1], e = _exact_rows(st, st["q"][b:b + 1], k, v, n - 1, start, 0)
            if weights is not None:
                w = weights[blocks].transpose(0, 1).flatten(1)
                w[:, n - 1] = 0
                w[:, :n] += e[:, 0].unflatten(0, (case["hkv"], -1)).sum(1)
                weights[blocks] = w.unflatten(1, (-1, BS)).transpose(0, 1)
        return (out, weights) if case["weights"] else out
    row = key = 0
    for b, n in enumerate(lens):
        total = n + case["cached"]
        if case["paged"]:
            blocks = st["block_tables"][b, :-(-total // BS)].long()
            k, v = (c[blocks].flatten(0, 1)[:total] for c in (st["k_cache"], st["v_cache"]))
        else:
            k, v = st["k"][key:key + total], st["v"][key:key + total]
        starts = none.expand(n) if st["key_starts"] is None else st["key_starts"][row:row + n].long()
        for a in range(0, n, 1024):
            z = min(n, a + 1024)
            out[row + a:row + z] = _exact_rows(st, st["q"][row + a:row + z], k, v, case["cached"] + a, starts[a:z],
                                               case["prefix"])[0]
        row, key = row + n, key + total
    return out
