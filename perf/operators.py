"""Cases of the 4-bit paged KV cache: writing it, reading it back, and attention over it.

The cache holds, for each (token, kv head), 128 codes of 4 bits and, for each
of its 4 groups of 32 dims, a scale s and a minimum z in fp16; a code c stands
for s * c + z. One uint8 tensor [num_blocks, num_kv_heads, 16, 1280] for K and
one for V: a 256-token block is 16 tiles of 16 tokens, a tile 16 x 64 bytes of
codes, then 16 x 4 x (s, z).

  K row: byte 16 t + 4 j + i holds dims 32 j + 8 t + 2 i (low nibble) and + 1.
  V row: 8-byte chunk r ^ (4 if token & 4 else 0), byte 2 j + i of it, holds
         dims 32 j + 4 r + 2 i (low nibble) and + 1.

Kinds of cases:
  "write_read"  rows quantised into their slots, then read back
  "read"        cached tokens read back into rows
  "decode"      one query token for each sequence
  "step"        the new tokens' rows written, then decode over them in one call;
                the rows that the step wrote come back as values beside its output
  "prefill"     causal attention of new tokens whose keys all sit in the cache
"""
import math
import random

import torch

own = False

D, BS, TILE, GROUP = 128, 256, 16, 32
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---- cases ----------------------------------------------------------------------------


def listed():
    return [
        # the smallest decode step: 4 sequences around one and two blocks; a call's latency
        dict(name="decode_tiny", kind="decode", dtype="bf16", hq=16, hkv=8, lens="37,256,300,511", pad=0,
             max_context=4096),
        # a serving batch: 256 sequences, contexts uniform in 512..4096
        dict(name="decode_batch", kind="decode", dtype="bf16", hq=16, hkv=8, seqs=256, lo=512, hi=4096, lens_seed=2,
             pad=0, max_context=4096),
        # the largest batch, long-tailed contexts (most far below the declared maximum), replayed with padding rows
        dict(name="decode_long_tailed", kind="decode", dtype="fp16", hq=16, hkv=8, seqs=512, mean=800, hi=4096,
             lens_seed=5, pad=24, max_context=4096),
        # one user with a long context: few rows, a long axis to split; 4 query heads to a kv head
        dict(name="decode_one_long", kind="decode", dtype="bf16", hq=32, hkv=8, lens="40007", pad=0,
             max_context=40960),
        # a small serving step with ragged contexts from a single token on, and padding rows
        dict(name="step_small", kind="step", dtype="fp16", hq=16, hkv=8, seqs=14, lo=1, hi=2500, lens_seed=3, pad=2,
             max_context=4096),
        # a serving step of 256 sequences
        dict(name="step_batch", kind="step", dtype="bf16", hq=16, hkv=8, seqs=256, lo=512, hi=4096, lens_seed=4,
             pad=0, max_context=4096),
        # the new rows of a decode step of 256 sequences: one token to a block
        dict(name="write_read_step", kind="write_read", dtype="bf16", hq=16, hkv=8, seqs=256, lo=1, hi=4096,
             lens_seed=6, new="last"),
        # a call of prompts of 100..1024 tokens, just below 16384 tokens
        dict(name="write_read_prompts", kind="write_read", dtype="bf16", hq=16, hkv=8, seqs=29, lo=100, hi=1024,
             lens_seed=7, new="all"),
        # one cached prefix of odd length read back for a chunk's contiguous attention
        dict(name="read_one_prefix", kind="read", dtype="fp16", hq=16, hkv=8, lens="1537", prefix=0),
        # 128 sequences behind one shared prefix of 1024 tokens, read back whole
        dict(name="read_shared_prefix", kind="read", dtype="bf16", hq=16, hkv=8, seqs=128, lo=64, hi=512,
             lens_seed=4, prefix=1024),
        # the prefix-hit call: 128 sequences behind a shared prefix of 1024 tokens, suffixes of 64..512 tokens
        dict(name="prefill_shared_prefix", kind="prefill", dtype="bf16", hq=16, hkv=8, seqs=128, lo=64, hi=512,
             lens_seed=4, prefix=1024),
        # a chunk of a long prompt: 5000 new tokens behind 7001 cached ones
        dict(name="prefill_chunk", kind="prefill", dtype="fp16", hq=16, hkv=8, lens="5000", prefix=7001),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "step", "write_read", "read", "prefill"])
    dtype = rng.choice(["bf16", "fp16"])
    seed = rng.randrange(1 << 30)
    if kind in ("decode", "step"):
        # at most 590,000 cached tokens, the size of the largest listed batch
        hq, hkv = rng.choice([(16, 8), (16, 8), (32, 8), (8, 8), (12, 6), (4, 1)])
        seqs = _log_int(rng, 1, 512)
        hi = max(1, min(_log_int(rng, 8, 40000), 590000 // seqs))
        return dict(kind=kind, dtype=dtype, hq=hq, hkv=hkv, seqs=seqs, lo=max(1, hi // rng.randint(1, 8)), hi=hi,
                    lens_seed=seed, pad=rng.choice([0, 0, 1, 9]), max_context=hi + rng.choice([0, 1, 1000]))
    if kind == "write_read":
        seqs = _log_int(rng, 1, 256)
        hi = max(1, min(_log_int(rng, 1, 4096), 32768 // seqs))
        return dict(kind=kind, dtype=dtype, hq=16, hkv=rng.choice([8, 8, 2, 5]), seqs=seqs, lo=max(1, hi // 3),
                    hi=hi, lens_seed=seed, new=rng.choice(["last", "all", "all"]))
    if kind == "read":
        seqs = _log_int(rng, 1, 64)
        return dict(kind=kind, dtype=dtype, hq=16, hkv=rng.choice([8, 8, 2, 5]), seqs=seqs, lo=1,
                    hi=_log_int(rng, 1, 2000), lens_seed=seed, prefix=rng.choice([0, 256, 1024]))
    seqs = _log_int(rng, 1, 96)
    hi = max(1, min(_log_int(rng, 1, 3000), 26000 // seqs))
    return dict(kind=kind, dtype=dtype, hq=16, hkv=8, seqs=seqs, lo=max(1, hi // 4), hi=hi, lens_seed=seed,
                prefix=rng.choice([0, 1, 300, 1024, 2500]) if seqs <= 32 else rng.choice([0, 513, 1024]))


def _lens(case):
    """The sequences' own lengths (without a shared prefix or padding rows), the same for every seed."""
    if "lens" in case:
        return [int(x) for x in case["lens"].split(",")]
    rng = random.Random(case["lens_seed"])
    if "mean" in case:
        return [max(1, min(case["hi"], 1 + int(rng.expovariate(1.0 / case["mean"])))) for _ in range(case["seqs"])]
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


# ---- the format, in elementary operations -----------------------------------------------


def _quantise(x):
    """Rows [..., 128] -> (codes [..., 128] uint8, params [..., 4, 2] fp16). The scale is computed in 32 bits; a
    code in 64, where the border between two codes is decided."""
    g = x.float().unflatten(-1, (4, GROUP))
    mn, mx = g.amin(-1), g.amax(-1)
    z = mn.half()
    s = ((mx - mn) / 15.0).half()
    sd = s.double().unsqueeze(-1)
    y = (g.double() - z.double().unsqueeze(-1)) / torch.where(sd > 0, sd, torch.ones_like(sd))
    codes = torch.where(sd > 0, y.round().clamp(0, 15), torch.zeros_like(y))
    return codes.to(torch.uint8).flatten(-2), torch.stack((s, z), -1)


def _pack(nibbles):
    return nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)


def _pack_k(codes):
    """[..., 128] codes -> [..., 64] bytes of a K row (dims ordered j, t, p -> t, j, p)."""
    return _pack(codes.unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-3))


def _pack_v(codes, token):
    """[N, H, 128] codes of tokens `token` (place in the tile, [N]) -> [N, H, 64] bytes of V rows."""
    rows = codes.unflatten(-1, (4, 8, 4)).transpose(-3, -2).flatten(-3)      # chunk r, group j, p
    return torch.where((token & 4).bool()[:, None, None], _pack(rows.roll(64, -1)), _pack(rows))


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _values(codes, params):
    """Codes [..., 128] and params [..., 4, 2] -> values in 32 bits."""
    p = params.float()
    return (codes.unflatten(-1, (4, GROUP)).float() * p[..., 0:1] + p[..., 1:2]).flatten(-2)


def _params(rows):
    return rows.contiguous().view(torch.float16).unflatten(-1, (4, 2))


def _unpack_k(b, params):
    return _values(_nibbles(b).unflatten(-1, (4, 4, 8)).transpose(-3, -2).flatten(-3), params)


def _unpack_v(b, params, token):
    """`token`: place in the tile, of a shape that broadcasts over b's leading dims and its last."""
    b = torch.where((token & 4).bool(), b.roll(32, -1), b)
    return _values(_nibbles(b).unflatten(-1, (8, 4, 4)).transpose(-3, -2).flatten(-3), params)


def _cells(cache):
    """Views of a cache's code rows [blocks, heads, 16, 16, 64] and parameter rows [blocks, heads, 16, 16, 16]."""
    return cache[..., :TILE * 64].unflatten(-1, (TILE, 64)), cache[..., TILE * 64:].unflatten(-1, (TILE, 16))


def _write_rows(rows, cache, slots, is_v):
    codes, params = _quantise(rows)
    blk, tile, tok = slots // BS, slots % BS // TILE, slots % TILE
    c, p = _cells(cache)
    c[blk, :, tile, tok] = _pack_v(codes, tok) if is_v else _pack_k(codes)
    p[blk, :, tile, tok] = params.flatten(-2).view(torch.uint8)


def _read_rows(cache, slots, is_v):
    blk, tile, tok = slots // BS, slots % BS // TILE, slots % TILE
    c, p = _cells(cache)
    b, q = c[blk, :, tile, tok], _params(p[blk, :, tile, tok])
    return _unpack_v(b, q, tok[:, None, None]) if is_v else _unpack_k(b, q)


def _read_blocks(cache, tables, is_v):
    """[B, W] block ids -> [B, W * 256, heads, 128] values in 32 bits."""
    c, p = _cells(cache[tables])                                             # [B, W, H, 16, 16, .]
    tok = torch.arange(TILE, device=cache.device)[:, None]
    v = _unpack_v(c, _params(p), tok) if is_v else _unpack_k(c, _params(p))
    return v.permute(0, 1, 3, 4, 2, 5).flatten(1, 3)


# ---- states -----------------------------------------------------------------------------


def _normal(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _filled_cache(blocks, hkv, gen):
    """A cache of quantised N(0, 1) rows: records of a smaller one in random order (every block differs)."""
    n = min(blocks * hkv, 256)
    cache = torch.empty((2, n, 1, BS // TILE, 1280), dtype=torch.uint8, device="cuda")
    slots = torch.arange(n * BS, device="cuda")
    for i in range(2):
        _write_rows(_normal((n * BS, 1, D), gen, torch.bfloat16), cache[i], slots, i == 1)
    pick = torch.randint(n, (2, blocks * hkv), generator=gen, device="cuda")
    return [cache[i, pick[i], 0].unflatten(0, (blocks, hkv)) for i in range(2)]


def _tables(lens, prefix, rng):
    """Block tables (host lists) of sequences behind a shared prefix, and the size of a pool with some spare blocks."""
    shared = prefix // BS
    need = shared + sum(-(-(prefix + n) // BS) - shared for n in lens)
    order = list(range(need + 16))
    rng.shuffle(order)
    tables, at = [], shared
    for n in lens:
        more = -(-(prefix + n) // BS) - shared
        tables.append(order[:shared] + order[at:at + more])
        at += more
    return tables, len(order)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    lens, dtype, hq, hkv = _lens(case), DTYPES[case["dtype"]], case["hq"], case["hkv"]
    prefix = case.get("prefix", 0)
    tables, blocks = _tables(lens, prefix, rng)
    st = dict(case=case, dtype=dtype, scale=1.0 / math.sqrt(D))
    k_cache, v_cache = _filled_cache(blocks, hkv, gen)
    st.update(k_cache=k_cache, v_cache=v_cache)

    def dev(a, dt=torch.int32):
        return torch.tensor(a, dtype=dt, device="cuda")

    def slots(table, first, last):
        return [table[p // BS] * BS + p % BS for p in range(first, last)]

    def qkv(n):
        # views of one fused projection, as attention layers get them
        t = _normal((n, (hq + 2 * hkv) * D), gen, dtype)
        return (t[:, :hq * D].unflatten(1, (hq, D)), t[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D)),
                t[:, (hq + hkv) * D:].unflatten(1, (hkv, D)))

    kind = case["kind"]
    if kind in ("decode", "step"):
        pad = case["pad"]
        width = -(-max(case["max_context"], max(lens)) // BS)
        st["live"] = len(lens)
        st["block_tables"] = dev([t + [-1] * (width - len(t)) for t in tables] + [[-1] * width] * pad)
        st["context_lens"] = dev(lens + [0] * pad)
        st["max_context"] = max(case["max_context"], max(lens))
        st["q"], st["k"], st["v"] = qkv(len(lens) + pad)
        st["slots"] = dev([slots(t, n - 1, n)[0] for t, n in zip(tables, lens)] + [-1] * pad)
        st["width"] = -(-max(lens) // BS)
    elif kind == "prefill":
        width = -(-(prefix + max(lens)) // BS)
        st["block_tables"] = dev([t + [-1] * (width - len(t)) for t in tables])
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu_q"] = dev(cu)
        st["cu_k"] = dev([c + prefix * i for i, c in enumerate(cu)])
        st["max_q"], st["max_k"] = max(lens), prefix + max(lens)
        st["q"] = qkv(cu[-1])[0]
        st["width"] = width
    else:
        first = [n - 1 if case.get("new") == "last" else 0 for n in lens]
        st["slots"] = dev([s for t, n, f in zip(tables, lens, first) for s in slots(t, f, prefix + n)])
        st["live"] = st["slots"].numel()
        if kind == "write_read":
            _, st["k"], st["v"] = qkv(st["live"])
    if kind in ("write_read", "read", "step"):
        n = st["slots"].numel()
        st["k_out"] = torch.zeros((n, hkv, D), dtype=dtype, device="cuda")
        st["v_out"] = torch.zeros_like(st["k_out"])
    return st


# ---- one pass ---------------------------------------------------------------------------


def run(st):
    kind, dtype = st["case"]["kind"], st["dtype"]
    kc, vc = st["k_cache"], st["v_cache"]
    if own:
        import paged_kv_cache_kvh_gb300 as pkv
        f16 = dtype == torch.float16
        if kind == "write_read":
            store = pkv.pkv_store_kvcache_q4_f16 if f16 else pkv.pkv_store_kvcache_q4
            store(st["k"], st["v"], kc, vc, st["slots"])
        if kind in ("decode", "step"):
            if "workspace" not in st:  # kept by the engine for all its steps
                st["workspace"] = pkv.decode_q4_workspace(st["q"].shape[0], st["max_context"], st["case"]["hq"],
                                                          st["case"]["hkv"])
            args = (kc, vc, st["block_tables"], st["context_lens"], st["max_context"], st["scale"], st["workspace"])
            if kind == "decode":
                return (pkv.pkv_decode_q4_f16 if f16 else pkv.pkv_decode_q4)(st["q"], *args)
            step = pkv.pkv_store_decode_q4_f16 if f16 else pkv.pkv_store_decode_q4
            out = step(st["q"], st["k"], st["v"], st["slots"], *args)
        if kind == "prefill":
            prefill = pkv.pkv_prefill_varlen_q4_f16 if f16 else pkv.pkv_prefill_varlen_q4
            return prefill(st["q"], st["cu_q"], st["cu_k"], st["max_q"], st["max_k"], st["scale"], kc, vc,
                           st["block_tables"])
        load = pkv.pkv_load_kvcache_q4_f16 if f16 else pkv.pkv_load_kvcache_q4
        rows = load(kc, vc, st["slots"], k=st["k_out"], v=st["v_out"])
        return rows if kind != "step" else (out, *rows)
    if kind == "decode":
        return _decode(st)
    if kind == "prefill":
        return _prefill(st)
    live = st["live"]
    at = st["slots"][:live].long()
    if kind in ("write_read", "step"):
        _write_rows(st["k"][:live], kc, at, False)
        _write_rows(st["v"][:live], vc, at, True)
    st["k_out"][:live] = _read_rows(kc, at, False)
    st["v_out"][:live] = _read_rows(vc, at, True)
    rows = (st["k_out"], st["v_out"])
    return rows if kind != "step" else (_decode(st), *rows)


def _softmax_rows(x):
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _decode(st):
    """One query for each sequence; rows without context give zeros."""
    live, hq, hkv = st["live"], st["case"]["hq"], st["case"]["hkv"]
    tables = st["block_tables"][:live, :st["width"]].long().clamp(min=0)
    q = st["q"][:live].float().unflatten(1, (hkv, hq // hkv))
    s = torch.einsum("bhgd,bthd->bhgt", q, _read_blocks(st["k_cache"], tables, False)) * st["scale"]
    there = torch.arange(s.shape[-1], device=s.device) < st["context_lens"][:live, None]
    p = _softmax_rows(s.masked_fill(~there[:, None, None], float("-inf")))
    out = torch.zeros_like(st["q"], memory_format=torch.contiguous_format)
    out[:live] = torch.einsum("bhgt,bthd->bhgd", p, _read_blocks(st["v_cache"], tables, True)).flatten(1, 2)
    return out


def _prefill(st):
    """Sequences padded to the longest; query row i of a sequence sits at position Lk - Lq + i."""
    hq, hkv, cu_q, cu_k = st["case"]["hq"], st["case"]["hkv"], st["cu_q"].long(), st["cu_k"].long()
    tables = st["block_tables"].long().clamp(min=0)
    lq, lk = cu_q.diff(), cu_k.diff()
    rows = torch.arange(st["q"].shape[0], device=cu_q.device)
    seq = torch.searchsorted(cu_q, rows, right=True) - 1
    i = torch.arange(st["max_q"], device=cu_q.device)
    take = (cu_q[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][take].float().unflatten(2, (hkv, hq // hkv))                  # [B, Lq, hkv, g, d]
    s = torch.einsum("bihgd,bthd->bhgit", q, _read_blocks(st["k_cache"], tables, False)) * st["scale"]
    t = torch.arange(s.shape[-1], device=s.device)
    seen = t <= torch.minimum(lk - lq + i[:, None], lk - 1).T[..., None]      # [B, Lq, T]
    p = _softmax_rows(s.masked_fill_(~seen[:, None, None], float("-inf")))
    o = torch.einsum("bhgit,bthd->bihgd", p, _read_blocks(st["v_cache"], tables, True)).flatten(2, 3)
    return o[seq, rows - cu_q[seq]].to(st["dtype"])


# ---- what a pass cannot do without --------------------------------------------------------


def work(case):
    lens, hq, hkv, prefix = _lens(case), case["hq"], case["hkv"], case.get("prefix", 0)
    cell, row = 2 * 80 * hkv, 2 * 2 * D * hkv                # K and V of a token: cached, and as 16-bit rows
    kind = case["kind"]
    if kind in ("write_read", "read"):
        n = len(lens) if case.get("new") == "last" else sum(lens) + prefix * len(lens)
        if kind == "write_read":
            return {"bytes": n * (row + cell + 4) + n * (cell + row + 4), "flops": 0}
        return {"bytes": (sum(lens) + prefix) * cell + n * (row + 4), "flops": 0}
    if kind == "prefill":
        pairs = sum(n * prefix + n * (n + 1) // 2 for n in lens)
        return {"bytes": (sum(lens) + prefix) * cell + 2 * sum(lens) * hq * D * 2, "flops": 4 * D * hq * pairs}
    b = len(lens) + case["pad"]
    moved = sum(lens) * cell + 2 * b * hq * D * 2 + 4 * (b + sum(-(-n // BS) for n in lens))
    if kind == "step":
        moved += len(lens) * (row + cell + 4) + len(lens) * (cell + row + 4)
    return {"bytes": moved, "flops": 4 * D * hq * sum(lens)}


# ---- the definition in 64 bits --------------------------------------------------------------


def _exact_quantised(x):
    """What rows [N, H, 128] read back as, in 64 bits: the stored scale and minimum are fp16 by definition."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for j in range(0, D, GROUP):
        g = x[..., j:j + GROUP].double()
        lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
        z, s = lo.to(torch.float16).double(), ((hi - lo) / 15).to(torch.float16).double()
        code = torch.nan_to_num((g - z) / s).round().clamp(0, 15)
        out[..., j:j + GROUP] = s * code + z
    return out


def _exact_gather(cache, block, token, is_v):
    """Values [n, H, 128] in 64 bits of the tokens (block, place in the block), dim by dim from the format's text."""
    tile, tok = token // TILE, token % TILE
    raw = cache[block, :, tile]                                               # [n, H, 1280]
    out = torch.empty((*raw.shape[:2], D), dtype=torch.float64, device=cache.device)
    for d in range(D):
        j = d // 32
        if is_v:
            r, p = d % 32 // 4, d % 4
            at = tok * 64 + (r ^ ((tok & 4))) * 8 + 2 * j + p // 2
        else:
            t, p = d % 32 // 8, d % 8
            at = tok * 64 + 16 * t + 4 * j + p // 2
        byte = raw.gather(2, at[:, None, None].expand(-1, raw.shape[1], 1))[..., 0].long()
        code = (byte >> (4 * (p % 2))) & 15
        where = 1024 + tok * 16 + 4 * j
        par = raw.gather(2, (where[:, None] + torch.arange(4, device=cache.device))[:, None].expand(-1, raw.shape[1], 4))
        s, z = par.contiguous().view(torch.float16).double().unbind(-1)
        out[..., d] = code * s + z
    return out


def _exact_attention(q, k, v, first, scale, group):
    """Rows [n, hq, 128] at positions first, first + 1, ... over keys [T, hkv, 128], in 64 bits."""
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    s = torch.einsum("nhd,thd->hnt", q.double(), k) * scale
    at = first + torch.arange(q.shape[0], device=q.device)
    s = s.masked_fill(torch.arange(k.shape[0], device=q.device) > at[:, None], float("-inf"))
    return torch.einsum("hnt,thd->nhd", torch.softmax(s, -1), v)


def exact(case, seed):
    st = prepare(case, seed)
    lens, hq, hkv, prefix, kind = _lens(case), case["hq"], case["hkv"], case.get("prefix", 0), case["kind"]
    slots = st["slots"].long() if "slots" in st else None
    if kind == "read":
        return tuple(_exact_gather(c, slots // BS, slots % BS, i == 1)
                     for i, c in enumerate((st["k_cache"], st["v_cache"])))
    if kind == "write_read":
        return _exact_quantised(st["k"]), _exact_quantised(st["v"])
    n_rows = st["q"].shape[0]
    out = torch.zeros((n_rows, hq, D), dtype=torch.float64, device="cuda")
    if kind == "step":
        new = [torch.zeros((n_rows, hkv, D), dtype=torch.float64, device="cuda") for _ in range(2)]
        for t, x in zip(new, (st["k"], st["v"])):
            t[:len(lens)] = _exact_quantised(x[:len(lens)])
    row = 0
    for b, n in enumerate(lens):
        total = prefix + n
        pos = torch.arange(total, device="cuda")
        block = st["block_tables"][b].long()[pos // BS]
        k, v = (_exact_gather(c, block, pos % BS, i == 1) for i, c in enumerate((st["k_cache"], st["v_cache"])))
        if kind == "step":
            k[-1], v[-1] = new[0][b], new[1][b]
        count = n if kind == "prefill" else 1
        out[row:row + count] = _exact_attention(st["q"][row:row + count], k, v, total - count, st["scale"], hq // hkv)
        row += count
    return (out, *new) if kind == "step" else out
