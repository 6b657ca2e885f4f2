"""The operators of a drafted (speculative) round on a paged KV cache, as timed cases.

Four operators stand around the cache's store and attention calls:

  qk_norm_rope   RMS norm of every query and key head and the position rotation, in one pass,
                 with the rotated K and the V written to their cache slots or K to a buffer
  plan_slots     block tables, slot maps, positions and prefix sums from request lengths
  tree_masks     ancestor bit masks and positions of drafted trees from their parent links
  tree_decode    attention of every drafted token over its request's cached tokens and its ancestors

Each case is a call of one of them; `own` chooses between plain torch operations and the package's
kernels. Lengths come from the case alone (its `layout` number), so that every seed has the same
shapes; values, trees, block placement and positions come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

HEAD_DIM = 128
MAX_POSITION = 36864   # rows of the angle table: the longest context of the cases and a tree behind it
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one request's draft of 8 tokens on a small model: latency is all there is
        {"name": "norm_rope_8_tokens", "op": "norm_rope", "tokens": 8, "hq": 8, "hkv": 2, "head_dim": 128,
         "rotary": 128, "interleaved": False, "norm": True, "store": False, "bs": 16, "skip": 0},
        # a round of drafts of 64 requests, an interleaved rotation of half of each head, no head norm
        {"name": "rope_interleaved_1021_tokens", "op": "norm_rope", "tokens": 1021, "hq": 16, "hkv": 8,
         "head_dim": 128, "rotary": 64, "interleaved": True, "norm": False, "store": False, "bs": 16, "skip": 0},
        # a decode round of 512 requests, padded rows among them: rotate and store
        {"name": "norm_rope_store_512_tokens", "op": "norm_rope", "tokens": 512, "hq": 32, "hkv": 8,
         "head_dim": 128, "rotary": 128, "interleaved": False, "norm": True, "store": True, "bs": 16, "skip": 9},
        # a full prefill round of 16384 tokens
        {"name": "norm_rope_store_16384_tokens", "op": "norm_rope", "tokens": 16384, "hq": 32, "hkv": 8,
         "head_dim": 128, "rotary": 128, "interleaved": False, "norm": True, "store": True, "bs": 16, "skip": 0},
        # one token for each of 512 running requests
        {"name": "plan_decode_512", "op": "plan_slots", "seqs": 512, "ctx": "lognormal", "ctx_lo": 16, "ctx_hi": 4096,
         "new_lo": 1, "new_hi": 1, "bs": 16, "pad": 0, "layout": 1},
        # chunks of 512 new tokens for 32 requests, and a batch padded to a captured size
        {"name": "plan_prefill_32x512", "op": "plan_slots", "seqs": 32, "ctx": "uniform", "ctx_lo": 0, "ctx_hi": 3584,
         "new_lo": 512, "new_hi": 512, "bs": 16, "pad": 100, "layout": 2},
        # one request's tree of 64 drafts
        {"name": "masks_1x64", "op": "tree_masks", "seqs": 1, "tree_lo": 64, "tree_hi": 64, "layout": 3},
        # ragged trees of 512 requests
        {"name": "masks_512_u1_64", "op": "tree_masks", "seqs": 512, "tree_lo": 1, "tree_hi": 64, "layout": 4},
        # one request of 5000 cached tokens and 8 drafts on a small model: latency of a split context
        {"name": "tree_1x8_ctx5000", "op": "tree_decode", "seqs": 1, "ctx": "uniform", "ctx_lo": 5000, "ctx_hi": 5000,
         "tree_lo": 8, "tree_hi": 8, "hq": 8, "hkv": 2, "bs": 16, "layout": 5},
        # a small model's round: 64 requests, 16 drafts each, large blocks
        {"name": "tree_64x16_u128_4096", "op": "tree_decode", "seqs": 64, "ctx": "uniform", "ctx_lo": 128,
         "ctx_hi": 4096, "tree_lo": 16, "tree_hi": 16, "hq": 16, "hkv": 8, "bs": 256, "layout": 6},
        # a large round: 256 requests of lognormal lengths with ragged trees
        {"name": "tree_256_u1_32_lognormal", "op": "tree_decode", "seqs": 256, "ctx": "lognormal", "ctx_lo": 16,
         "ctx_hi": 4096, "tree_lo": 1, "tree_hi": 32, "hq": 32, "hkv": 8, "bs": 16, "layout": 7},
        # long contexts with wide trees: 64 drafts x 4 heads a KV head
        {"name": "tree_8x64_ctx32768", "op": "tree_decode", "seqs": 8, "ctx": "uniform", "ctx_lo": 32768,
         "ctx_hi": 32768, "tree_lo": 64, "tree_hi": 64, "hq": 32, "hkv": 8, "bs": 256, "layout": 8},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "plan_slots", "tree_masks", "tree_decode", "tree_decode"))
    if op == "norm_rope":
        hkv, group = rng.choice((1, 2, 3, 4, 6, 8)), rng.choice((1, 2, 3, 4, 5, 8))
        dim = rng.choice((64, 128, 128, 256))
        most = max(1, 16384 * 48 * 128 // ((group + 2) * hkv * dim))
        tokens = _log_int(rng, 1, min(16384, most))
        return {"op": op, "tokens": tokens, "hq": hkv * group, "hkv": hkv, "head_dim": dim,
                "rotary": rng.choice((dim, dim, dim // 2, 16)), "interleaved": rng.random() < 0.3,
                "norm": rng.random() < 0.7, "store": rng.random() < 0.6, "bs": rng.choice((1, 8, 16, 24, 256)),
                "skip": rng.choice((0, 0, 7))}
    layout = rng.randrange(1 << 30)
    if op == "plan_slots":
        seqs = _log_int(rng, 1, 512)
        new_hi = _log_int(rng, 1, max(1, min(2048, 16384 // seqs)))
        return {"op": op, "seqs": seqs, "ctx": rng.choice(("uniform", "lognormal")), "ctx_lo": rng.choice((0, 16)),
                "ctx_hi": _log_int(rng, 17, 4096), "new_lo": rng.choice((0, 1, new_hi)), "new_hi": new_hi,
                "bs": rng.choice((1, 7, 16, 32, 256)), "pad": rng.choice((0, 0, 33)), "layout": layout}
    if op == "tree_masks":
        seqs = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, 128 if seqs <= 128 else 64)
        return {"op": op, "seqs": seqs, "tree_lo": rng.choice((0, 1, hi)), "tree_hi": hi, "layout": layout}
    hkv, group = rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 3, 4, 4, 5, 8, 16))
    hi = _log_int(rng, 1, 100)
    ctx_hi = _log_int(rng, 17, 32768)
    # bounded by the largest listed cases: cached bytes, score entries
    most = min(256, 8 * 32768 * 8 // (ctx_hi * hkv), 8 * 32768 * 64 * 32 // (ctx_hi * hi * hkv * group))
    return {"op": op, "seqs": _log_int(rng, 1, max(1, most)), "ctx": rng.choice(("uniform", "lognormal")),
            "ctx_lo": rng.choice((0, 1, 16)), "ctx_hi": ctx_hi, "tree_lo": rng.choice((1, hi)), "tree_hi": hi,
            "hq": hkv * group, "hkv": hkv, "bs": rng.choice((1, 6, 8, 16, 16, 48, 256)), "layout": layout}


def _lengths(case, what):
    """The case's own list of lengths: `ctx` cached tokens, `new` tokens or `tree` nodes of each request."""
    rng = random.Random("%s %d" % (what, case["layout"]))
    out = []
    for _ in range(case["seqs"]):
        if what == "ctx" and case["ctx"] == "lognormal":
            x = int(round(math.exp(math.log(800.0) + rng.gauss(0.0, 1.0))))
            out.append(max(case["ctx_lo"], min(case["ctx_hi"], x)))
        else:
            out.append(rng.randint(case[what + "_lo"], case[what + "_hi"]))
    if what == "tree" and not any(out):
        out[0] = 1
    return out


# ---------------------------------------------------------------- inputs --

def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int64).astype(np.int32))).cuda()


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _prefix(lens):
    return np.concatenate([[0], np.cumsum(np.asarray(lens, dtype=np.int64))])


def _parents(rs, lens):
    """Parent of each node (index in its own tree, -1: a child of the last cached token), most of them recent."""
    out = []
    for n in lens:
        t = np.arange(n)
        out.append(np.maximum(-1, t - 1 - np.floor(rs.exponential(2.0, n)).astype(np.int64)))
    return np.concatenate(out) if out else np.zeros(0, np.int64)


def _mask_words(parents, lens, words):
    bits = []
    row = 0
    for n in lens:
        m = np.zeros((n, words * 32), np.uint8)
        for t in range(n):
            p = int(parents[row + t])
            if p >= 0:
                m[t] = m[p]
            m[t, t] = 1
        bits.append(m)
        row += n
    packed = np.packbits(np.concatenate(bits), axis=1, bitorder="little")
    return np.ascontiguousarray(packed).view("<i4")


def _place(rs, blocks_of, num_blocks, width):
    """Block tables: every request's blocks at random places of the pool, -1 behind them."""
    perm = rs.permutation(num_blocks)
    table = np.full((len(blocks_of), max(1, width)), -1, np.int64)
    at = 0
    for i, n in enumerate(blocks_of):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, perm[at:]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rs = np.random.RandomState(int(seed) % (1 << 32))
    s = {"op": case["op"]}
    if case["op"] == "norm_rope":
        t, hq, hkv, d, r = case["tokens"], case["hq"], case["hkv"], case["head_dim"], case["rotary"]
        # q, k and v are views into the projection's fused output
        qkv = _normal(gen, t, (hq + 2 * hkv) * d)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        s["q_weight"] = (1 + 0.1 * _normal(gen, d).float()).to(torch.bfloat16) if case["norm"] else None
        s["k_weight"] = (1 + 0.1 * _normal(gen, d).float()).to(torch.bfloat16) if case["norm"] else None
        s["positions"] = _i32(rs.randint(0, MAX_POSITION, t))
        angle = torch.arange(MAX_POSITION, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["interleaved"] = case["interleaved"]
        s["store"] = case["store"]
        if case["store"]:
            bs = case["bs"]
            nb = -(-t * 5 // (4 * bs)) + 1
            s["k_cache"], s["v_cache"] = _normal(gen, nb, bs, hkv, d), _normal(gen, nb, bs, hkv, d)
            slots = rs.permutation(nb * bs)[:t]
            if case["skip"]:
                slots[::case["skip"]] = -1
            s["slot_mapping"] = _i32(slots)
        return s
    if case["op"] == "plan_slots":
        ctx, new, bs = _lengths(case, "ctx"), _lengths(case, "new"), case["bs"]
        have = [-(-c // bs) for c in ctx]
        need = [-(-(c + n) // bs) for c, n in zip(ctx, new)]
        num_blocks = -(-sum(need) * 5 // 4) + 8
        s["block_tables"], free = (_i32(a) for a in _place(rs, have, num_blocks, (max(need) + 31) // 32 * 32))
        s["free_blocks"] = free
        s["free_cursor"] = _i32([rs.randint(0, 4)])
        s["context_lens"], s["new_lens"] = _i32(ctx), _i32(new)
        s["bs"], s["num_blocks"] = bs, num_blocks
        s["max_tokens"] = max(1, sum(new) + case["pad"])
        return s
    trees = _lengths(case, "tree")
    s["cu_seqlens_q"] = _i32(_prefix(trees))
    s["max_seqlen_q"] = max(trees)
    words = (max(trees) + 31) // 32
    parents = _parents(rs, trees)
    if case["op"] == "tree_masks":
        s["parents"] = _i32(parents)
        s["context_lens"] = _i32(rs.randint(0, 32768, len(trees)))
        return s
    ctx, bs, hq, hkv = _lengths(case, "ctx"), case["bs"], case["hq"], case["hkv"]
    blocks = [-(-c // bs) for c in ctx]
    num_blocks = sum(blocks) * 5 // 4 + 1
    table, _ = _place(rs, blocks, num_blocks, (max(blocks) + 31) // 32 * 32)
    total = sum(trees)
    s["block_tables"], s["context_lens"], s["max_context_len"] = _i32(table), _i32(ctx), max(ctx)
    s["k_cache"] = _normal(gen, num_blocks, bs, hkv, HEAD_DIM)
    s["v_cache"] = _normal(gen, num_blocks, bs, hkv, HEAD_DIM)
    qkv = _normal(gen, total, (hq + 2 * hkv) * HEAD_DIM)
    s["q"] = qkv[:, :hq * HEAD_DIM].unflatten(1, (hq, HEAD_DIM)).contiguous()
    s["key"] = qkv[:, hq * HEAD_DIM:(hq + hkv) * HEAD_DIM].unflatten(1, (hkv, HEAD_DIM))
    s["value"] = qkv[:, (hq + hkv) * HEAD_DIM:].unflatten(1, (hkv, HEAD_DIM))
    s["tree_mask"] = torch.from_numpy(_mask_words(parents, trees, words).copy()).cuda()
    s["scale"] = HEAD_DIM ** -0.5
    return s


# ------------------------------------------------------------------- run --

def run(s):
    return {"norm_rope": _norm_rope, "plan_slots": _plan_slots, "tree_masks": _tree_masks,
            "tree_decode": _tree_decode}[s["op"]](s)


def _norm_rope(s):
    if own:
        import paged_kv_cache_86_gb300 as pkv
        if s["store"]:
            q = pkv.qk_norm_rope_store(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slot_mapping"],
                                       s["positions"], s["cos_sin"], s["q_weight"], s["k_weight"], EPS,
                                       s["interleaved"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        q, k = pkv.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["q_weight"], s["k_weight"], EPS,
                                s["interleaved"])
        return {"q": q, "k": k}
    rows = s["cos_sin"][s["positions"].long()]
    half = rows.shape[1] // 2
    cos, sin = rows[:, None, :half], rows[:, None, half:]

    def rotated(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        part, rest = x[..., :2 * half], x[..., 2 * half:]
        if s["interleaved"]:
            a, b = part[..., 0::2], part[..., 1::2]
            part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = part[..., :half], part[..., half:]
            part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([part, rest], -1).to(torch.bfloat16)

    q, k = rotated(s["q"], s["q_weight"]), rotated(s["k"], s["k_weight"])
    if not s["store"]:
        return {"q": q, "k": k}
    kept = (s["slot_mapping"] >= 0).nonzero()[:, 0]
    slots = s["slot_mapping"].long()[kept]
    s["k_cache"].flatten(0, 1)[slots] = k[kept]
    s["v_cache"].flatten(0, 1)[slots] = s["v"][kept]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plan_slots(s):
    if own:
        import paged_kv_cache_86_gb300 as pkv
        p = pkv.plan_slots(s["context_lens"], s["new_lens"], s["block_tables"], s["free_blocks"], s["free_cursor"],
                           s["bs"], s["num_blocks"], s["max_tokens"])
        return {"slot_mapping": p.slot_mapping, "positions": p.positions, "cu_seqlens_q": p.cu_seqlens_q,
                "cu_seqlens_k": p.cu_seqlens_k, "context_lens": p.context_lens, "free_cursor": p.free_cursor,
                "block_tables": s["block_tables"]}
    ctx, new, bs = s["context_lens"].long(), s["new_lens"].long(), s["bs"]
    after = ctx + new
    have, need = (ctx + bs - 1) // bs, (after + bs - 1) // bs
    zero = torch.zeros(1, dtype=torch.int64, device=ctx.device)
    taken = torch.cat([zero, torch.cumsum(need - have, 0)])
    cu_q, cu_k = torch.cat([zero, torch.cumsum(new, 0)]), torch.cat([zero, torch.cumsum(after, 0)])
    col = torch.arange(s["block_tables"].shape[1], device=ctx.device)[None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    at = (s["free_cursor"].long() + taken[:-1])[:, None] + col - have[:, None]
    ids = s["free_blocks"][at.clamp(0, s["free_blocks"].numel() - 1)]
    s["block_tables"].copy_(torch.where(fresh, ids, s["block_tables"]))
    t = torch.arange(s["max_tokens"], device=ctx.device)
    seq = torch.searchsorted(cu_q[1:], t, right=True)
    real = seq < ctx.numel()
    seq = seq.clamp(max=ctx.numel() - 1)
    pos = torch.where(real, ctx[seq] + t - cu_q[seq], 0)
    slot = s["block_tables"][seq, (pos // bs).clamp(max=col.numel() - 1)].long() * bs + pos % bs
    out = {"slot_mapping": torch.where(real, slot, -1), "positions": pos, "cu_seqlens_q": cu_q, "cu_seqlens_k": cu_k,
           "context_lens": after, "free_cursor": s["free_cursor"].long() + taken[-1:]}
    out = {k: v.to(torch.int32) for k, v in out.items()}
    out["block_tables"] = s["block_tables"]
    return out


def _tree_masks(s):
    if own:
        import paged_kv_cache_86_gb300 as pkv
        mask, positions = pkv.tree_masks(s["parents"], s["cu_seqlens_q"], s["context_lens"], s["max_seqlen_q"])
        return {"tree_mask": mask, "positions": positions}
    n, words = s["parents"].numel(), (s["max_seqlen_q"] + 31) // 32
    row = torch.arange(n, device=s["parents"].device)
    seq = torch.searchsorted(s["cu_seqlens_q"][1:].long(), row, right=True)
    first = s["cu_seqlens_q"].long()[seq]
    at = torch.where(s["parents"] >= 0, first + s["parents"].long(), n)   # row n: above every root
    # ancestors by doubling: after k steps every row holds its nearest 2^k ancestors and jumps 2^k up
    seen = torch.zeros(n + 1, words * 32, dtype=torch.bool, device=row.device)
    seen[row, row - first] = True
    at = torch.cat([at, torch.full((1,), n, device=row.device)])
    for _ in range(max(1, (s["max_seqlen_q"] - 1).bit_length())):
        seen = seen | seen[at]
        at = at[at]
    seen = seen[:n]
    weight = 2 ** torch.arange(32, device=row.device, dtype=torch.int64)
    mask = (seen.unflatten(1, (words, 32)).long() * weight).sum(-1)
    mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(torch.int32)
    return {"tree_mask": mask, "positions": (s["context_lens"].long()[seq] + seen.sum(1) - 1).to(torch.int32)}


def _tree_decode(s):
    if own:
        import paged_kv_cache_86_gb300 as pkv
        return pkv.tree_decode(s["q"], s["key"], s["value"], s["k_cache"], s["v_cache"], s["block_tables"],
                               s["context_lens"], s["cu_seqlens_q"], s["tree_mask"], s["scale"], s["max_seqlen_q"],
                               s["max_context_len"])
    q, dev = s["q"], s["q"].device
    (total, hq, d), (_, bs, hkv, _) = q.shape, s["k_cache"].shape
    cu, ctx = s["cu_seqlens_q"].long(), s["context_lens"].long()
    seqs, most, long = ctx.numel(), s["max_seqlen_q"], s["max_context_len"]
    # every request padded to the longest context and the widest tree
    pos = torch.arange(long, device=dev)
    cached = pos[None] < ctx[:, None]
    slot = torch.where(cached, s["block_tables"].long()[:, pos // bs] * bs + pos % bs, 0)
    u = torch.arange(most, device=dev)
    real = u[None] < (cu[1:] - cu[:-1])[:, None]
    row = torch.where(real, cu[:-1, None] + u, 0)

    def heads(cache, fresh):   # [S, Hkv, long + most, D] in 32 bits
        return torch.cat([cache.flatten(0, 1)[slot], fresh[row]], 1).float().permute(0, 2, 1, 3)

    qs = q[row].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.matmul(qs, heads(s["k_cache"], s["key"]).transpose(2, 3)) * s["scale"]
    bit = (s["tree_mask"].long()[row][:, :, u // 32] >> (u % 32)) & 1
    seen = torch.cat([cached[:, None].expand(-1, most, -1), (bit != 0) & real[:, None]], 2)
    seen = seen[:, None, :, None].expand(-1, -1, -1, hq // hkv, -1).flatten(2, 3)
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score.sub_(torch.where(top > -math.inf, top, 0.0)))
    total_weight = weight.sum(-1, keepdim=True)
    o = torch.matmul(weight, heads(s["v_cache"], s["value"])) / torch.where(total_weight > 0, total_weight, 1.0)
    o = o.unflatten(2, (most, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    t = torch.arange(total, device=dev)
    seq = torch.searchsorted(cu[1:], t, right=True)
    return o[seq, t - cu[seq]].to(torch.bfloat16)


# ------------------------------------------------------------------ work --

def work(case):
    if case["op"] == "norm_rope":
        t, d = case["tokens"], case["head_dim"]
        heads = case["hq"] + case["hkv"]
        moved = heads + (case["hkv"] if case["store"] else 0)
        # the angle row of a token and its position and slot
        return {"bytes": 2 * t * moved * d * 2 + t * (case["rotary"] * 4 + 8),
                "flops": t * heads * ((4 * d if case["norm"] else 0) + 3 * case["rotary"])}
    if case["op"] == "plan_slots":
        ctx, new, bs = _lengths(case, "ctx"), _lengths(case, "new"), case["bs"]
        fresh = sum(-(-(c + n) // bs) - -(-c // bs) for c, n in zip(ctx, new))
        tokens = sum(new) + case["pad"]
        return {"bytes": case["seqs"] * 20 + fresh * 8 + tokens * 8 + case["seqs"] * 4, "flops": 0}
    trees = _lengths(case, "tree")
    if case["op"] == "tree_masks":
        words = (max(trees) + 31) // 32
        return {"bytes": sum(trees) * (8 + 4 * words) + case["seqs"] * 8, "flops": 0}
    ctx, hq, hkv = _lengths(case, "ctx"), case["hq"], case["hkv"]
    rows = sum(trees)
    return {"bytes": (2 * sum(ctx) * hkv + 2 * rows * hkv + 2 * rows * hq) * HEAD_DIM * 2,
            "flops": 4 * HEAD_DIM * hq * sum(t * (c + t) for t, c in zip(trees, ctx))}


# ----------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_norm_rope(s)
    if case["op"] == "tree_decode":
        return _exact_tree_decode(s)
    return None


def _exact_norm_rope(s):
    table = s["cos_sin"].double()
    half = table.shape[1] // 2
    turn = torch.complex(table[:, :half], table[:, half:]).index_select(0, s["positions"].long()).unsqueeze(1)

    def one(x, w):
        x = x.double()
        if w is not None:
            power = x.pow(2).sum(-1, keepdim=True) / x.shape[-1]
            x = x / (power + EPS).sqrt() * w.double()
        head = x[..., :2 * half].unflatten(-1, (half, 2) if s["interleaved"] else (2, half))
        z = torch.complex(head[..., 0], head[..., 1]) if s["interleaved"] else \
            torch.complex(head[..., 0, :], head[..., 1, :])
        z = z * turn
        head = torch.stack([z.real, z.imag], -1 if s["interleaved"] else -2).flatten(-2)
        return torch.cat([head, x[..., 2 * half:]], -1)

    q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
    if not s["store"]:
        return {"q": q, "k": k}
    caches = {}
    for name, rows in (("k_cache", k), ("v_cache", s["v"].double())):
        c = s[name].double()
        flat = c.view(-1, *c.shape[2:])
        ok = s["slot_mapping"] >= 0
        flat.index_copy_(0, s["slot_mapping"][ok].long(), rows[ok])
        caches[name] = c
    return {"q": q, **caches}


def _exact_tree_decode(s):
    (total, hq, d), (_, bs, hkv, _) = s["q"].shape, s["k_cache"].shape
    group = hq // hkv
    out = torch.zeros(total, hq, d, dtype=torch.float64, device=s["q"].device)
    cu, ctx = s["cu_seqlens_q"].tolist(), s["context_lens"].tolist()
    words = s["tree_mask"].cpu().numpy().view(np.uint32)
    for i, n in enumerate(ctx):
        a, b = cu[i], cu[i + 1]
        if a == b:
            continue
        blocks = s["block_tables"][i, :-(-n // bs)].long()
        keys = torch.cat([s["k_cache"][blocks].flatten(0, 1)[:n], s["key"][a:b]]).double()
        values = torch.cat([s["v_cache"][blocks].flatten(0, 1)[:n], s["value"][a:b]]).double()
        bits = np.unpackbits(words[a:b].view(np.uint8), axis=1, bitorder="little")[:, :b - a]
        hidden = torch.zeros(b - a, n + b - a, dtype=torch.bool, device=out.device)
        hidden[:, n:] = torch.from_numpy(bits == 0).to(out.device)
        for h in range(hq):
            score = s["q"][a:b, h].double() @ keys[:, h // group].T * s["scale"]
            score[hidden] = -math.inf
            out[a:b, h] = torch.softmax(score, -1) @ values[:, h // group]
    return out
