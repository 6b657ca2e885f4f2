"""Long contexts at fewer bytes on a paged KV cache, as timed cases.

Five operators:

  store     new K/V rows of a round into an fp8 E4M3 cache with one scale per (block, KV head)
  load      the requests' rows of that cache, back in bf16
  decode8   one query per request over that cache, whole or behind a sliding window with sinks
  decode    one query per request over the bf16 cache behind a sliding window with sinks
  prefill   query chunks over the bf16 cache behind a sliding window with sinks

A sliding window of w with s sinks leaves position t the keys p <= t with p < s or p > t - w.

Each case is a call of one of them; `own` chooses between plain torch operations and the package's
kernels. Lengths come from the case alone (its `layout` number), so that every seed has the same
shapes; values and block placement come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

HEAD_DIM = 128
E4M3_MAX = 448.0
E4M3 = torch.float8_e4m3fn
SCALE_EXP = (-120, 119)   # exponents of the power-of-two scales


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a decode round of 512 requests: one new token each into partly filled blocks
        {"name": "store_decode_512", "op": "store", "seqs": 512, "ctx": "lognormal", "ctx_lo": 16, "ctx_hi": 4096,
         "new_lo": 1, "new_hi": 1, "hkv": 8, "bs": 16, "layout": 1},
        # a prefill round: chunks of 512 tokens of 32 requests behind ragged prefixes
        {"name": "store_prefill_32x512", "op": "store", "seqs": 32, "ctx": "uniform", "ctx_lo": 0, "ctx_hi": 3584,
         "new_lo": 512, "new_hi": 512, "hkv": 8, "bs": 16, "layout": 2},
        # three requests of a small model read back
        {"name": "load_300_5000_70", "op": "load", "seqs": 3, "ctx": "three", "ctx_lo": 70, "ctx_hi": 5000, "hkv": 2,
         "bs": 16, "layout": 3},
        # a whole batch's history read back before a prefill round over it
        {"name": "load_256_lognormal", "op": "load", "seqs": 256, "ctx": "lognormal", "ctx_lo": 16, "ctx_hi": 4096,
         "hkv": 8, "bs": 16, "layout": 4},
        # three requests of a small model: latency is all there is
        {"name": "decode8_300_5000_70", "op": "decode8", "seqs": 3, "ctx": "three", "ctx_lo": 70, "ctx_hi": 5000,
         "window": 0, "sinks": 0, "hq": 8, "hkv": 2, "bs": 16, "layout": 5},
        # a full decode round of 512 requests of lognormal lengths
        {"name": "decode8_512_lognormal", "op": "decode8", "seqs": 512, "ctx": "lognormal", "ctx_lo": 16,
         "ctx_hi": 4096, "window": 0, "sinks": 0, "hq": 32, "hkv": 8, "bs": 16, "layout": 6},
        # long contexts, large blocks, an odd group of query heads, the last 4096 tokens and 4 sinks
        {"name": "decode8_64x32768_w4096", "op": "decode8", "seqs": 64, "ctx": "uniform", "ctx_lo": 32768,
         "ctx_hi": 32768, "window": 4096, "sinks": 4, "hq": 40, "hkv": 8, "bs": 256, "layout": 7},
        # a small model's round behind a short window
        {"name": "decode_64_u128_4096_w512", "op": "decode", "seqs": 64, "ctx": "uniform", "ctx_lo": 128,
         "ctx_hi": 4096, "window": 512, "sinks": 4, "hq": 16, "hkv": 8, "bs": 256, "layout": 8},
        # a large round of long contexts behind a window of 1024
        {"name": "decode_512_w1024", "op": "decode", "seqs": 512, "ctx": "lognormal", "ctx_lo": 16, "ctx_hi": 4096,
         "window": 1024, "sinks": 64, "hq": 32, "hkv": 8, "bs": 16, "layout": 9},
        # one ragged chunk behind a long prefix: latency
        {"name": "prefill_1x130_ctx5000_w512", "op": "prefill", "seqs": 1, "ctx": "uniform", "ctx_lo": 5000,
         "ctx_hi": 5000, "new_lo": 130, "new_hi": 130, "window": 512, "sinks": 4, "hq": 8, "hkv": 2, "bs": 16,
         "layout": 10},
        # a prefill round of 16384 tokens behind prefixes of up to 3584
        {"name": "prefill_32x512_w1024", "op": "prefill", "seqs": 32, "ctx": "uniform", "ctx_lo": 0, "ctx_hi": 3584,
         "new_lo": 512, "new_hi": 512, "window": 1024, "sinks": 4, "hq": 32, "hkv": 8, "bs": 16, "layout": 11},
        # long prompts in chunks of 4096, a window of 4096
        {"name": "prefill_4x4096_ctx28672_w4096", "op": "prefill", "seqs": 4, "ctx": "uniform", "ctx_lo": 28672,
         "ctx_hi": 28672, "new_lo": 4096, "new_hi": 4096, "window": 4096, "sinks": 64, "hq": 32, "hkv": 8,
         "bs": 256, "layout": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("store", "load", "decode8", "decode8", "decode", "decode", "prefill", "prefill"))
    case = {"op": op, "ctx": rng.choice(("uniform", "lognormal")), "bs": rng.choice((1, 6, 8, 16, 16, 24, 48, 256)),
            "layout": rng.randrange(1 << 30)}
    hkv = rng.choice((1, 2, 3, 4, 6, 8))
    if op == "store":
        seqs = _log_int(rng, 1, 512)
        new_hi = _log_int(rng, 1, max(1, min(2048, 16384 // seqs)))
        return case | {"seqs": seqs, "ctx_lo": rng.choice((0, 16)), "ctx_hi": _log_int(rng, 17, 4096),
                       "new_lo": rng.choice((0, 1, new_hi)), "new_hi": new_hi, "hkv": hkv}
    if op == "load":
        ctx_hi = _log_int(rng, 17, 32768)
        return case | {"seqs": _log_int(rng, 1, min(512, 250_000 * 8 // (ctx_hi * hkv))), "ctx_lo": rng.choice((0, 1)),
                       "ctx_hi": ctx_hi, "hkv": hkv}
    group = rng.choice((1, 2, 3, 4, 4, 5, 7, 8, 12, 16))
    windowed = op != "decode8" or rng.random() < 0.5
    case |= {"window": _log_int(rng, 1, 8192) if windowed else 0,
             "sinks": rng.choice((0, 1, 4, 64, 300)) if windowed else 0, "hkv": hkv, "hq": hkv * group}
    if op != "prefill":
        ctx_hi = _log_int(rng, 17, 32768)
        seen = min(ctx_hi, case["window"] + case["sinks"]) if windowed else ctx_hi
        most = min(512, 250_000 * 8 // (seen * hkv), 2_000_000 * 32 // (seen * hkv * group),
                   2_500_000 * 8 // (ctx_hi * hkv))
        return case | {"seqs": _log_int(rng, 1, max(1, most)), "ctx_lo": rng.choice((0, 1, 16)), "ctx_hi": ctx_hi}
    new_hi = _log_int(rng, 1, 4096)
    ctx_hi = _log_int(rng, 17, 28672)
    seen = min(ctx_hi + new_hi, case["window"] + case["sinks"] + new_hi)
    most = min(32, 16384 // new_hi, 4 * 4096 * 8192 * 32 // (new_hi * seen * hkv * group),
               2_500_000 * 8 // (ctx_hi * hkv))
    return case | {"seqs": _log_int(rng, 1, max(1, most)), "ctx_lo": rng.choice((0, 1, 16)), "ctx_hi": ctx_hi,
                   "new_lo": rng.choice((1, new_hi)), "new_hi": new_hi}


def _lengths(case, what):
    """The case's own list of lengths: `ctx` cached tokens or `new` tokens of each request."""
    if what == "ctx" and case["ctx"] == "three":
        return [300, 5000, 70]
    rng = random.Random("%s %d" % (what, case["layout"]))
    out = []
    for _ in range(case["seqs"]):
        if what == "ctx" and case["ctx"] == "lognormal":
            x = int(round(math.exp(math.log(800.0) + rng.gauss(0.0, 1.0))))
            out.append(max(case["ctx_lo"], min(case["ctx_hi"], x)))
        else:
            out.append(rng.randint(case[what + "_lo"], case[what + "_hi"]))
    if not any(out):
        out[0] = 1
    return out


def _totals(case):
    """Cached tokens of each request before the call, new ones, and both."""
    ctx = _lengths(case, "ctx")
    new = _lengths(case, "new") if case["op"] in ("store", "prefill") else [0] * len(ctx)
    return ctx, new, [c + n for c, n in zip(ctx, new)]


# ---------------------------------------------------------------- inputs --

def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int64).astype(np.int32))).cuda()


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _codes(gen, *shape):
    """E4M3 codes of a normal distribution that fills about a third of the type's range."""
    return (torch.randn(shape, generator=gen, device="cuda") * 100).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)


def _scales(gen, *shape):
    """Powers of two around the one that gives the codes' values a deviation of about one."""
    return torch.exp2(torch.randint(-8, -5, shape, generator=gen, device="cuda").float())


def _prefix(lens):
    return np.concatenate([[0], np.cumsum(np.asarray(lens, dtype=np.int64))])


def _place(rs, blocks_of, num_blocks):
    """Block tables: every request's blocks at random places of the pool, -1 behind them."""
    perm = rs.permutation(num_blocks)
    table = np.full((len(blocks_of), (max(blocks_of) + 31) // 32 * 32), -1, np.int64)
    at = 0
    for i, n in enumerate(blocks_of):
        table[i, :n] = perm[at:at + n]
        at += n
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rs = np.random.RandomState(int(seed) % (1 << 32))
    op, hkv, bs = case["op"], case["hkv"], case["bs"]
    ctx, new, after = _totals(case)
    blocks = [-(-n // bs) for n in after]
    num_blocks = sum(blocks) * 5 // 4 + 1
    s = {"op": op, "block_tables": _i32(_place(rs, blocks, num_blocks)), "max_context_len": max(after)}
    if op in ("store", "load", "decode8"):
        s["k_cache"], s["v_cache"] = _codes(gen, num_blocks, bs, hkv, HEAD_DIM), _codes(gen, num_blocks, bs, hkv, HEAD_DIM)
        s["k_scales"], s["v_scales"] = _scales(gen, num_blocks, hkv), _scales(gen, num_blocks, hkv)
    else:
        s["k_cache"], s["v_cache"] = _normal(gen, num_blocks, bs, hkv, HEAD_DIM), _normal(gen, num_blocks, bs, hkv, HEAD_DIM)
    s["context_lens"] = _i32(after)
    if op == "load":
        s["row_starts"], s["num_rows"] = _i32(_prefix(after)[:-1]), sum(after)
        return s
    if op == "store":
        # key and value are views into the projection's fused output; a few tokens are larger than the rest
        total = sum(new)
        size = torch.exp(0.7 * torch.randn(total, 1, generator=gen, device="cuda"))
        kv = (torch.randn(total, 2 * hkv * HEAD_DIM, generator=gen, device="cuda") * size).to(torch.bfloat16)
        s["key"] = kv[:, :hkv * HEAD_DIM].unflatten(1, (hkv, HEAD_DIM))
        s["value"] = kv[:, hkv * HEAD_DIM:].unflatten(1, (hkv, HEAD_DIM))
        s["cu_seqlens_q"], s["max_seqlen_q"] = _i32(_prefix(new)), max(new)
        return s
    s["window"], s["sinks"], s["scale"] = case["window"], case["sinks"], HEAD_DIM ** -0.5
    s["q"] = _normal(gen, sum(new) if op == "prefill" else len(ctx), case["hq"], HEAD_DIM)
    if op == "prefill":
        s["cu_seqlens_q"], s["cu_seqlens_k"] = _i32(_prefix(new)), _i32(_prefix(after))
        s["max_seqlen_q"] = max(new)
    return s


# ------------------------------------------------------------------- run --

def run(s):
    return {"store": _store, "load": _load, "decode8": _decode8, "decode": _decode, "prefill": _prefill}[s["op"]](s)


def _store(s):
    if own:
        import paged_kv_cache_86_gb300 as pkv
        pkv.store_kvcache_fp8_block(s["key"], s["value"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                    s["block_tables"], s["cu_seqlens_q"], s["context_lens"])
        return _stored(s)
    cu, after, bs = s["cu_seqlens_q"].long(), s["context_lens"].long(), s["k_cache"].shape[1]
    start = after - (cu[1:] - cu[:-1])
    # every request padded to the most blocks that its new tokens can touch
    most = (s["max_seqlen_q"] + bs - 2) // bs + 1
    dev = cu.device
    block = start[:, None] // bs + torch.arange(most, device=dev)                        # [S, most]
    touched = (block * bs < after[:, None]) & (after > start)[:, None]
    block, seq = block[touched], touched.nonzero()[:, 0]                                  # [U]
    ids = s["block_tables"][seq, block].long()
    pos = block[:, None] * bs + torch.arange(bs, device=dev)                              # [U, bs]
    fresh = (pos >= start[seq, None]) & (pos < after[seq, None])
    older = pos < start[seq, None]
    row = torch.where(fresh, cu[seq, None] + pos - start[seq, None], 0)
    for x, cache, scales in ((s["key"], s["k_cache"], s["k_scales"]), (s["value"], s["v_cache"], s["v_scales"])):
        x = x[row].float()                                                                # [U, bs, Hkv, D]
        held = cache[ids].view(E4M3).float() * scales[ids][:, None, :, None]
        top = torch.where(fresh[..., None, None] & x.isfinite(), x.abs(), 0.0).amax((1, 3))   # [U, Hkv]
        part, exp = torch.frexp(top)
        exp = torch.where(part * 2 <= E4M3_MAX / 256, exp - 9, exp - 8).clamp(*SCALE_EXP)
        scale = torch.exp2(torch.where(top > 0, exp, SCALE_EXP[0]).float())
        scale = torch.where(older.any(1)[:, None], torch.maximum(scale, scales[ids]), scale)
        value = torch.where(fresh[..., None, None], x, held) / scale[:, None, :, None]
        code = value.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
        kept = (fresh | older)[..., None, None]
        cache[ids] = torch.where(kept, code, cache[ids])
        scales[ids] = scale
    return _stored(s)


def _stored(s):
    return {"k_cache": s["k_cache"].view(E4M3), "v_cache": s["v_cache"].view(E4M3), "k_scales": s["k_scales"],
            "v_scales": s["v_scales"]}


def _load(s):
    if own:
        import paged_kv_cache_86_gb300 as pkv
        key, value = pkv.load_kvcache_fp8_block(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                                s["block_tables"], s["context_lens"], s["row_starts"], s["num_rows"])
        return {"key": key, "value": value}
    first, bs = s["row_starts"].long(), s["k_cache"].shape[1]
    row = torch.arange(s["num_rows"], device=first.device)
    seq = torch.searchsorted(first, row, right=True) - 1
    pos = row - first[seq]
    ids = s["block_tables"][seq, pos // bs].long()
    slot = ids * bs + pos % bs
    return {name: (cache.flatten(0, 1)[slot].view(E4M3).float() * scales[ids][..., None]).to(torch.bfloat16)
            for name, cache, scales in (("key", s["k_cache"], s["k_scales"]), ("value", s["v_cache"], s["v_scales"]))}


def _hidden_before(first_row, s):
    """How many keys behind the sinks the first row (at these positions) and so every later one leaves out."""
    if not s["window"]:
        return torch.zeros_like(first_row)
    return (first_row + 1 - s["window"] - s["sinks"]).clamp(min=0)


def _gathered(s, shift, count, most):
    """Positions [S, most] of the keys that are not left out, which of them are real, and K and V [S, Hkv, most, D]
    in 32 bits."""
    bs = s["k_cache"].shape[1]
    j = torch.arange(most, device=shift.device)
    real = j[None] < count[:, None]
    pos = torch.where(real, j + (j >= s["sinks"]) * shift[:, None], 0)
    ids = torch.where(real, s["block_tables"].gather(1, pos // bs).long(), 0)
    slot = ids * bs + pos % bs

    def rows(cache, scales):
        x = cache.flatten(0, 1)[slot]
        x = x.float() if scales is None else x.view(E4M3).float().mul_(scales[ids][..., None])
        return x.masked_fill_(~real[..., None, None], 0.0).permute(0, 2, 1, 3)

    return pos, real, rows(s["k_cache"], s.get("k_scales")), rows(s["v_cache"], s.get("v_scales"))


def _attended(q, keys, values, seen, scale):
    """q [S, Hkv, rows, D]; seen [S, 1, rows, most]; a row that sees nothing gives zeros."""
    score = torch.matmul(q, keys.transpose(2, 3)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = weight.sum(-1, keepdim=True)
    return torch.matmul(weight, values) / torch.where(total > 0, total, 1.0)


def _one_token(s):
    hq, hkv, ctx = s["q"].shape[1], s["k_cache"].shape[2], s["context_lens"].long()
    shift = _hidden_before(ctx - 1, s)
    most = min(s["max_context_len"], s["window"] + s["sinks"]) if s["window"] else s["max_context_len"]
    _, real, keys, values = _gathered(s, shift, ctx - shift, most)
    q = s["q"].float().unflatten(1, (hkv, hq // hkv))
    o = _attended(q, keys, values, real[:, None, None], s["scale"])
    return o.flatten(1, 2).to(torch.bfloat16)


def _decode8(s):
    if own:
        import paged_kv_cache_86_gb300 as pkv
        return pkv.paged_decode_fp8_block(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                          s["block_tables"], s["context_lens"], s["scale"], window=s["window"],
                                          sinks=s["sinks"], max_context_len=s["max_context_len"])
    return _one_token(s)


def _decode(s):
    if own:
        import paged_kv_cache_86_gb300 as pkv
        return pkv.paged_decode_window(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                                       s["scale"], s["window"], s["sinks"], max_context_len=s["max_context_len"])
    return _one_token(s)


def _prefill(s):
    if own:
        import paged_kv_cache_86_gb300 as pkv
        return pkv.paged_prefill_window(s["q"], s["k_cache"], s["v_cache"], s["cu_seqlens_q"], s["cu_seqlens_k"],
                                        s["block_tables"], s["scale"], s["window"], s["sinks"], s["max_seqlen_q"],
                                        s["max_context_len"])
    hq, hkv, cu, after = s["q"].shape[1], s["k_cache"].shape[2], s["cu_seqlens_q"].long(), s["context_lens"].long()
    new, rows = cu[1:] - cu[:-1], s["max_seqlen_q"]
    shift = _hidden_before(after - new, s)
    most = min(s["max_context_len"], s["window"] + s["sinks"] + rows - 1)
    pos, real, keys, values = _gathered(s, shift, after - shift, most)
    u = torch.arange(rows, device=cu.device)
    at = (after - new)[:, None] + u                                                       # [S, rows]
    q = s["q"][torch.where(u[None] < new[:, None], cu[:-1, None] + u, 0)].float()         # [S, rows, Hq, D]
    q = q.unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    near = pos[:, None] > at[..., None] - s["window"]
    seen = real[:, None] & (pos[:, None] <= at[..., None]) & (near | (pos[:, None] < s["sinks"]))
    seen = seen[:, None, :, None].expand(-1, -1, -1, hq // hkv, -1).flatten(2, 3)
    o = _attended(q, keys, values, seen, s["scale"])
    o = o.unflatten(2, (rows, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    t = torch.arange(s["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    return o[seq, t - cu[seq]].to(torch.bfloat16)


# ------------------------------------------------------------------ work --

def _seen(case, last):
    """Keys that a row at position `last` sees."""
    n = last + 1
    return min(n, case["window"] + case["sinks"]) if case["window"] else n


def work(case):
    ctx, new, after = _totals(case)
    hkv, bs = case["hkv"], case["bs"]
    row = hkv * HEAD_DIM
    if case["op"] == "store":
        scales = sum(-(-a // bs) - c // bs for c, n, a in zip(ctx, new, after) if n) * hkv * 4
        return {"bytes": 2 * (sum(new) * row * 3 + scales), "flops": 0}
    scales = sum(-(-a // bs) for a in after) * hkv * 4
    if case["op"] == "load":
        return {"bytes": 2 * (sum(after) * row * 3 + scales), "flops": 0}
    if case["op"] == "prefill":
        rows = sum(new)
        keys = sum(min(a, _seen(case, c) + n - 1) for c, n, a in zip(ctx, new, after) if n)
        pairs = sum(_seen(case, c + r) for c, n in zip(ctx, new) for r in range(n))
        return {"bytes": 2 * keys * row * 2 + 2 * rows * case["hq"] * HEAD_DIM * 2,
                "flops": 4 * HEAD_DIM * case["hq"] * pairs}
    keys = sum(_seen(case, c - 1) for c in ctx)
    held = 2 if case["op"] == "decode" else 1
    if held == 1:
        scales = sum(-(-_seen(case, c - 1) // bs) for c in ctx) * hkv * 4
    return {"bytes": 2 * keys * row * held + (2 * scales if held == 1 else 0) + 2 * len(ctx) * case["hq"] * HEAD_DIM * 2,
            "flops": 4 * HEAD_DIM * case["hq"] * keys}


# ----------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "load": _exact_load}.get(case["op"], _exact_attention)(s)


def _e4m3_grid():
    """The finite E4M3 values by code, from the format's fields."""
    out = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = math.ldexp(m / 8, -6) if e == 0 else math.ldexp(1 + m / 8, e - 7)
        out.append(-v if code & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _exact_store(s):
    """Request by request and block by block; a value goes to the nearest of the format's 127 magnitudes."""
    grid = _e4m3_grid()
    size = grid[:127]
    middle = (size[1:] + size[:-1]) / 2
    cu, after, table = s["cu_seqlens_q"].tolist(), s["context_lens"].tolist(), s["block_tables"].tolist()
    bs = s["k_cache"].shape[1]

    def nearest(v):
        m = v.abs().clamp(max=E4M3_MAX)
        lo = torch.bucketize(m, middle)                       # m <= middle[lo]
        tie = (lo < 126) & (m == middle[lo.clamp(max=125)])   # to the even code
        lo = torch.where(tie & (lo % 2 == 1), lo + 1, lo)
        return torch.copysign(size[lo], v)

    jobs, rows_of = {}, {}   # by block: how many older rows it has, and (offset, row) of its new ones
    for i, a in enumerate(after):
        start = a - (cu[i + 1] - cu[i])
        for p in range(start, a):
            b = table[i][p // bs]
            jobs.setdefault(b, max(0, start - p // bs * bs))
            rows_of.setdefault(b, []).append((p % bs, cu[i] + p - start))
    out = {}
    for x, cache, scales, name in ((s["key"], s["k_cache"], s["k_scales"], "k"), (s["value"], s["v_cache"], s["v_scales"], "v")):
        held, scale = grid[cache.long()], scales.double()
        ids = list(jobs)
        owner = torch.tensor([k for k, b in enumerate(ids) for _ in rows_of[b]], device="cuda")
        offset = torch.tensor([o for b in ids for o, _ in rows_of[b]], device="cuda")
        row = torch.tensor([r for b in ids for _, r in rows_of[b]], device="cuda")
        older = torch.tensor([jobs[b] for b in ids], device="cuda")
        block = torch.tensor(ids, device="cuda")
        xd = x.double()[row]
        top = torch.zeros(len(ids), x.shape[1], dtype=torch.float64, device="cuda")
        top.index_reduce_(0, owner, xd.abs().amax(-1), "amax")
        need = torch.full_like(top, 2.0 ** SCALE_EXP[0])
        for e in range(SCALE_EXP[0], SCALE_EXP[1]):
            need = torch.where(top > E4M3_MAX * 2.0 ** e, 2.0 ** (e + 1), need)
        now = torch.where((older > 0)[:, None], torch.maximum(need, scale[block]), need)
        # older rows of the touched blocks in the new scale, then the new rows
        old_rows = torch.arange(bs, device="cuda")[None] < older[:, None]
        moved = nearest(held[block] * (scale[block] / now)[:, None, :, None])
        held[block] = torch.where(old_rows[..., None, None], moved, held[block])
        held[block[owner], offset] = nearest(xd / now[owner][..., None])
        scale[block] = now
        out[name + "_cache"], out[name + "_scales"] = held, scale
    return out


def _history(s, i, n):
    """The first n K and V rows of request i in 64 bits: [n, Hkv, D]."""
    bs = s["k_cache"].shape[1]
    blocks = s["block_tables"][i, :-(-n // bs)].long()
    out = []
    for c in ("k", "v"):
        x = s[c + "_cache"][blocks]
        x = _e4m3_grid()[x.long()] * s[c + "_scales"][blocks].double()[:, None, :, None] if c + "_scales" in s else x.double()
        out.append(x.flatten(0, 1)[:n])
    return out


def _exact_load(s):
    rows = [_history(s, i, n) for i, n in enumerate(s["context_lens"].tolist())]
    return {"key": torch.cat([k for k, _ in rows]), "value": torch.cat([v for _, v in rows])}


def _exact_attention(s):
    hq, hkv, window, sinks = s["q"].shape[1], s["k_cache"].shape[2], s["window"], s["sinks"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    after = s["context_lens"].tolist()
    cu = s["cu_seqlens_q"].tolist() if s["op"] == "prefill" else list(range(len(after) + 1))
    for i, n in enumerate(after):
        a, b = cu[i], cu[i + 1]
        if a == b or n == 0:
            continue
        first = max(0, n - (b - a) + 1 - window) if window else 0      # first key in any row's window
        front = min(sinks, first)
        keys, values = (torch.cat([x[:front], x[first:]]) for x in _history(s, i, n))
        p = torch.cat([torch.arange(front, device="cuda"), torch.arange(first, n, device="cuda")])
        t = torch.arange(n - (b - a), n, device="cuda")[:, None]
        hidden = p > t
        if window:
            hidden = hidden | ((p <= t - window) & (p >= sinks))
        for h in range(hkv):
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            score = torch.einsum("thd,pd->htp", s["q"][a:b, heads].double(), keys[:, h]) * s["scale"]
            score = score.masked_fill(hidden, -math.inf)
            out[a:b, heads] = torch.einsum("htp,pd->thd", torch.softmax(score, -1), values[:, h])
    return out
