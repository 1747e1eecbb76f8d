"""Measured cases of the paged serving operators: block tables and slot maps built
from request lengths, the block-scaled 8-bit KV writer, and grouped-query attention
over that cache (single tokens, chunks, capped / biased / masked scores).

listed() names the measured cases and draw() takes more from the same ranges.
prepare() makes a case's inputs from a seed, run() makes one pass over them: the
plain torch form, or with own = True the library's entry points.  work() counts the
bytes and operations no implementation can do without, exact() evaluates the
definitions in 64 bits.

The cache: blocks of 64 tokens, k_cache and v_cache [num_blocks, h_kv, 64, d] in e4m3
or int8, one float32 scale for each (block, head).  A key is code * scale.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 64
DEV = "cuda"


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of an ordinary batch: each request grows by one token
        {"name": "table_decode_b64", "op": "table", "batch": 64, "kv_len": 8192, "q_len": 1, "ragged": True},
        # a wave of prompts admitted at once beside running requests
        {"name": "table_prompts_b1000", "op": "table", "batch": 1000, "kv_len": 500, "q_len": 700, "ragged": True},
        # the writer behind one decode step
        {"name": "write_decode_b64", "op": "write", "batch": 64, "kv_len": 8192, "q_len": 1, "ragged": True,
         "h_kv": 8, "d": 128, "cache": "e4m3"},
        # the writer behind a wave of ragged prompts
        {"name": "write_prompts_int8", "op": "write", "batch": 16, "kv_len": 100, "q_len": 4096, "ragged": True,
         "h_kv": 8, "d": 128, "cache": "int8"},
        # the smallest call: a first reply token on a short prompt, where latency counts
        {"name": "decode_b1_77", "op": "attend", "batch": 1, "q_len": 1, "kv_len": 77, "ragged": False, "h_q": 32,
         "h_kv": 8, "d": 128, "cache": "e4m3", "causal": True, "softcap": 0.0, "alibi": False, "prefix": 0, "docs": 0},
        # an ordinary decode batch at the framework's benchmark lengths
        {"name": "decode_b64_8k", "op": "attend", "batch": 64, "q_len": 1, "kv_len": 8192, "ragged": False, "h_q": 64,
         "h_kv": 8, "d": 128, "cache": "e4m3", "causal": True, "softcap": 0.0, "alibi": False, "prefix": 0, "docs": 0},
        # a model with one KV head per query head, small heads, odd ragged lengths, distance bias
        {"name": "decode_mha_d64_int8", "op": "attend", "batch": 37, "q_len": 1, "kv_len": 5001, "ragged": True,
         "h_q": 16, "h_kv": 16, "d": 64, "cache": "int8", "causal": True, "softcap": 0.0, "alibi": True, "prefix": 0,
         "docs": 0},
        # one long conversation: the split over a long axis, capped scores
        {"name": "decode_b1_128k_cap", "op": "attend", "batch": 1, "q_len": 1, "kv_len": 131072, "ragged": False,
         "h_q": 64, "h_kv": 8, "d": 128, "cache": "int8", "causal": True, "softcap": 50.0, "alibi": False, "prefix": 0,
         "docs": 0},
        # four draft tokens of each request verified at once
        {"name": "verify_b32_sq4", "op": "attend", "batch": 32, "q_len": 4, "kv_len": 4096, "ragged": True, "h_q": 32,
         "h_kv": 8, "d": 128, "cache": "e4m3", "causal": True, "softcap": 0.0, "alibi": False, "prefix": 0, "docs": 0},
        # a long prompt's second half on top of its first
        {"name": "chunk_8k_on_8k", "op": "attend", "batch": 1, "q_len": 8192, "kv_len": 16384, "ragged": False,
         "h_q": 32, "h_kv": 8, "d": 128, "cache": "e4m3", "causal": True, "softcap": 0.0, "alibi": False, "prefix": 0,
         "docs": 0},
        # ragged prompts of packed documents, capped scores
        {"name": "prompts_docs_cap", "op": "attend", "batch": 6, "q_len": 4000, "kv_len": 4000, "ragged": True,
         "h_q": 32, "h_kv": 4, "d": 128, "cache": "int8", "causal": True, "softcap": 30.0, "alibi": False, "prefix": 0,
         "docs": 5},
        # ragged prompts whose first part sees itself in both directions, distance bias, small heads
        {"name": "prompts_prefix_alibi_d64", "op": "attend", "batch": 5, "q_len": 2500, "kv_len": 2900, "ragged": True,
         "h_q": 24, "h_kv": 8, "d": 64, "cache": "e4m3", "causal": True, "softcap": 0.0, "alibi": True, "prefix": 700,
         "docs": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "write", "attend", "attend", "attend", "attend"])
    cache = rng.choice(["e4m3", "int8"])
    d = rng.choice([64, 128])
    if op == "table":
        q = rng.choice([1, _log(rng, 2, 700)])
        return {"op": op, "batch": _log(rng, 1, 1000), "kv_len": _log(rng, 1, 8192), "q_len": q, "ragged": True}
    if op == "write":
        q = rng.choice([1, _log(rng, 2, 4096)])
        b = _log(rng, 1, 128 if q < 64 else max(1, 65536 // q // 2))
        return {"op": op, "batch": b, "kv_len": _log(rng, 1, 4096), "q_len": q, "ragged": rng.random() < 0.7,
                "h_kv": rng.choice([1, 2, 4, 8]), "d": d, "cache": cache}
    h_kv = rng.choice([1, 2, 4, 8])
    h_q = h_kv * rng.choice([1, 2, 4, 7, 8])
    mods = rng.choice(["none", "none", "softcap", "alibi", "prefix", "docs", "softcap+docs", "alibi+prefix", "full"])
    c = {"op": op, "h_q": h_q, "h_kv": h_kv, "d": d, "cache": cache, "ragged": rng.random() < 0.7,
         "causal": mods != "full", "softcap": rng.choice([20.0, 50.0]) if "softcap" in mods else 0.0,
         "alibi": "alibi" in mods, "docs": rng.randint(2, 9) if "docs" in mods else 0}
    if rng.random() < 0.5:  # single tokens and short runs of them
        c["q_len"] = rng.choice([1, 1, 1, rng.randint(2, 8)])
        c["batch"] = _log(rng, 1, 64)
        c["kv_len"] = max(c["q_len"], _log(rng, 16, min(131072, 524288 // c["batch"])))
    else:                   # chunks and whole prompts
        c["q_len"] = _log(rng, 17, 4096)
        c["batch"] = _log(rng, 1, max(1, min(16, 4096 // c["q_len"])))
        c["kv_len"] = c["q_len"] + rng.choice([0, _log(rng, 1, 8192)])
    c["prefix"] = rng.randint(1, c["kv_len"]) if "prefix" in mods else 0
    return c


# --------------------------------------------------------------------------- a case's lengths
def _lens(c):
    """(new tokens, length with them) of each request: fixed by the case, not by the seed."""
    b = c["batch"]
    r = np.random.RandomState((b * 1000003 + c["kv_len"] * 101 + c["q_len"]) % (1 << 31))
    if c["op"] == "attend":
        kv = np.full(b, c["kv_len"], np.int64)
        q = np.full(b, c["q_len"], np.int64)
        if c["ragged"]:
            u = r.uniform(0.1, 1.0, b)
            kv = np.maximum(1, np.round(kv * u).astype(np.int64))
            if c["q_len"] > 8:
                q = np.maximum(1, np.round(q * u).astype(np.int64))
            kv = np.maximum(kv, q)
        return q, kv
    old = np.full(b, c["kv_len"], np.int64)
    q = np.full(b, c["q_len"], np.int64)
    if c["ragged"]:
        old = np.round(old * r.uniform(0.0, 1.0, b)).astype(np.int64)
        if c["q_len"] > 1:
            q = np.round(q * r.uniform(0.0, 1.0, b)).astype(np.int64)
            q[0] = max(1, q[0])
    return q, old + q


def _doc_cuts(c):
    """Per request: the sorted first positions of its documents (the first is 0), and its length."""
    q, kv = _lens(c)
    r = np.random.RandomState((c["docs"] * 7919 + c["kv_len"]) % (1 << 31))
    return [np.unique(np.concatenate([[0], r.randint(0, n, max(0, c["docs"] - 1))])) for n in kv], kv


def _doc_bounds(c):
    q, _ = _lens(c)
    cuts, kv = _doc_cuts(c)
    out = []
    for r in range(c["batch"]):
        pos = np.arange(kv[r] - q[r], kv[r])
        at = np.searchsorted(cuts[r], pos, side="right") - 1
        ends = np.append(cuts[r][1:], kv[r])
        out.append(np.stack([cuts[r][at], ends[at]], 1))
    return np.concatenate(out).astype(np.int32)


def _visible(c):
    """(first, end) of the cache positions that each query token sees."""
    q, kv = _lens(c)
    lo, hi = [], []
    docs = _doc_bounds(c) if c["docs"] else None
    at = 0
    for r in range(c["batch"]):
        pos = np.arange(kv[r] - q[r], kv[r])
        e = np.full(q[r], kv[r])
        if c["causal"]:
            e = np.minimum(e, np.maximum(pos + 1, min(c["prefix"], kv[r])))
        s = np.zeros(q[r], np.int64)
        if docs is not None:
            d = docs[at:at + q[r]]
            s, e = d[:, 0].astype(np.int64), np.minimum(e, d[:, 1])
        at += q[r]
        lo.append(s)
        hi.append(np.maximum(s, e))
    return lo, hi


def work(c):
    q, kv = _lens(c)
    total = int(q.sum())
    if c["op"] == "table":
        old = kv - q
        grown = int((-(-kv // BLOCK) + (-old // BLOCK)).sum())
        # lengths in, lengths and offsets out, block numbers in and out, slots out
        return {"bytes": 8 * c["batch"] + 8 * c["batch"] + 8 * grown + 8 * total, "flops": 0}
    if c["op"] == "write":
        row = c["h_kv"] * c["d"]
        touched = int((-(-kv // BLOCK) - (kv - q) // BLOCK)[q > 0].sum())
        return {"bytes": 2 * (total * row * 3 + touched * c["h_kv"] * 4), "flops": 0}
    lo, hi = _visible(c)
    pairs = sum(int((h - s).sum()) for s, h in zip(lo, hi))
    tokens = sum(int(h.max() - s.min()) for s, h in zip(lo, hi) if len(h))
    return {"bytes": tokens * c["h_kv"] * 2 * (c["d"] + 4 / BLOCK) + total * c["h_q"] * (4 * c["d"] + 4),
            "flops": 4 * pairs * c["h_q"] * c["d"]}


# --------------------------------------------------------------------------- inputs
def _paging(kv, g, spare=3):
    """A table of blocks spread over a pool: [b, most blocks] int32, padded with 0."""
    need = -(-kv // BLOCK)
    total = int(need.sum())
    perm = torch.randperm(total + spare, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((len(kv), max(1, int(need.max()) + 1)), dtype=torch.int32, device=DEV)
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(need)])).to(DEV)
    need_t = torch.from_numpy(need).to(DEV)
    col = torch.arange(table.shape[1], device=DEV)
    at = first[:-1, None] + col[None]
    inside = col[None] < need_t[:, None]
    table = torch.where(inside, perm[at.clamp(max=total + spare - 1)], table)
    return table.contiguous(), perm, total + spare, total


def _codes(shape, cache, g):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if cache == "e4m3":
        return (x * 90).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return (x * 30).clamp_(-127, 127).round_().to(torch.int8)


def _scales(shape, cache, g):
    """Powers of two, as the writer leaves them, a few steps apart."""
    e = torch.randint(-1, 2, shape, generator=g, device=DEV)
    return torch.ldexp(torch.ones(shape, device=DEV), e - (7 if cache == "e4m3" else 5)).float()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    q, kv = _lens(c)
    total = int(q.sum())
    cu = _i32(np.concatenate([[0], np.cumsum(q)]))
    if c["op"] == "table":
        old = kv - q
        table, perm, pool, used = _paging(old, g)
        grown = int((-(-kv // BLOCK) - (-(-old // BLOCK))).sum())
        cols = int((-(-kv // BLOCK)).max()) + 2
        wide = torch.zeros((c["batch"], cols), dtype=torch.int32, device=DEV)
        n = min(cols, table.shape[1])
        wide[:, :n] = table[:, :n]
        free = (used + torch.randperm(grown + 17, generator=g, device=DEV)).to(torch.int32)
        return {"c": c, "block_table": wide, "cache_seqlens": _i32(old), "new_lens": _i32(q), "free_blocks": free,
                "num_free": torch.full((1,), grown + 17, dtype=torch.int32, device=DEV), "max_new_tokens": total}
    table, _, pool, _ = _paging(kv, g)
    h_kv, d = c["h_kv"], c["d"]
    s = {"c": c, "block_table": table, "cu": cu, "total": total,
         "k_cache": _codes((pool, h_kv, BLOCK, d), c["cache"], g),
         "v_cache": _codes((pool, h_kv, BLOCK, d), c["cache"], g),
         "k_scale": _scales((pool, h_kv), c["cache"], g), "v_scale": _scales((pool, h_kv), c["cache"], g)}
    if c["op"] == "write":
        s["cache_seqlens"], s["new_seqlens"] = _i32(kv - q), _i32(kv)
        # keys and values as they leave one fused projection: strided views of its rows
        kv_rows = torch.randn((total, 2, h_kv, d), generator=g, device=DEV)
        kv_rows *= torch.exp(0.5 * torch.randn((total, 2, h_kv, 1), generator=g, device=DEV))
        kv_rows = kv_rows.to(torch.bfloat16)
        s["k"], s["v"] = kv_rows[:, 0], kv_rows[:, 1]
        return s
    s["cache_seqlens"] = _i32(kv)
    s["max_q"], s["max_kv"] = int(q.max()), int(kv.max())
    s["q"] = torch.randn((total, c["h_q"], d), generator=g, device=DEV).to(torch.bfloat16)
    s["slopes"] = s["prefix"] = s["docs"] = None
    if c["alibi"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["h_q"] + 1, device=DEV) / c["h_q"]).float()
    if c["prefix"]:
        s["prefix"] = _i32(np.minimum(c["prefix"], kv))
    if c["docs"]:
        s["docs"] = _i32(_doc_bounds(c))
    return s


# --------------------------------------------------------------------------- plain forms
def _table_plain(s):
    old, new = s["cache_seqlens"].long(), s["new_lens"].long()
    table, free, have = s["block_table"], s["free_blocks"], s["num_free"].long()
    before, after = (old + BLOCK - 1) // BLOCK, (old + new + BLOCK - 1) // BLOCK
    need = after - before
    last = torch.cumsum(need, 0)
    granted = (need == 0) | (last <= have)
    need_ok = torch.where(granted, need, torch.zeros_like(need))
    col = torch.arange(table.shape[1], device=DEV)[None]
    fresh = (col >= before[:, None]) & (col < (before + need_ok)[:, None])
    at = have - 1 - ((last - need)[:, None] + col - before[:, None])
    table.copy_(torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table))
    cu = torch.zeros(old.numel() + 1, dtype=torch.int64, device=DEV)
    cu[1:] = torch.cumsum(new, 0)
    i = torch.arange(s["max_new_tokens"], device=DEV)
    r = torch.bucketize(i, cu[1:], right=True).clamp(max=old.numel() - 1)
    pos = old[r] + i - cu[r]
    slot = table[r, (pos // BLOCK).clamp(max=table.shape[1] - 1)].long() * BLOCK + pos % BLOCK
    slot = torch.where(granted[r] & (i < cu[-1]), slot, torch.full_like(slot, -1))
    return (slot, cu.to(torch.int32), torch.where(granted, old + new, old).to(torch.int32),
            (have - need_ok.sum()).to(torch.int32), table)


def _pow2_scale(amax, cache):
    """The smallest power of two at which amax fits the code range; 0 for amax 0."""
    m, e = torch.frexp(amax)
    top, bits = (0.875, 9) if cache == "e4m3" else (127.0 / 128.0, 7)
    k = torch.where(m <= top, e - bits, e - bits + 1).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), k), torch.zeros_like(amax))


def _to_codes(x, cache):
    if cache == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn)
    return x.round().clamp(-127, 127).to(torch.int8)


def _write_plain(s):
    c = s["c"]
    old, cu, table = s["cache_seqlens"].long(), s["cu"].long(), s["block_table"].long()
    i = torch.arange(s["total"], device=DEV)
    r = torch.bucketize(i, cu[1:], right=True)
    pos = old[r] + i - cu[r]
    block, row = table[r, pos // BLOCK], pos % BLOCK
    grows = (cu[1:] > cu[:-1]) & (old % BLOCK > 0)     # requests whose first written block holds older tokens
    first = table[torch.arange(old.numel(), device=DEV), old // BLOCK]
    held = torch.where(grows, old % BLOCK, torch.zeros_like(old))
    live = torch.zeros(s["k_scale"].shape[0], device=DEV).index_add(0, first, grows.float()) > 0
    touched = torch.zeros_like(live)
    touched[block] = True
    for x, codes, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x.float()
        amax = torch.zeros_like(scale).index_reduce(0, block, x.abs().amax(-1), "amax")
        was = torch.where(live[:, None], scale, torch.zeros_like(scale))
        now = torch.maximum(_pow2_scale(amax, c["cache"]), was)
        # older tokens of a block whose scale grew
        ratio = torch.where(now > 0, was / now, torch.ones_like(was))[first]
        f = codes.view(torch.int8)[first].view(codes.dtype).float()
        moved = _to_codes(f * ratio[:, :, None, None], c["cache"]).float()
        keep = (torch.arange(BLOCK, device=DEV)[None] < held[:, None])[:, None, :, None]
        f = torch.where(keep & (ratio < 1)[:, :, None, None], moved, f)
        at = first[grows]
        codes.view(torch.int8)[at] = _to_codes(f, c["cache"]).view(torch.int8)[grows]
        scale.copy_(torch.where(touched[:, None], now, scale))
        div = now[block][:, :, None]
        y = torch.where(div > 0, x / torch.where(div > 0, div, torch.ones_like(div)), torch.zeros_like(x))
        codes.view(torch.int8)[block, :, row] = _to_codes(y, c["cache"]).view(torch.int8)
    return s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]


def _attend_plain(s):
    c = s["c"]
    b, h_kv, d, g = c["batch"], c["h_kv"], c["d"], c["h_q"] // c["h_kv"]
    cu, kv = s["cu"].long(), s["cache_seqlens"].long()
    n_blk = -(-s["max_kv"] // BLOCK)
    table = s["block_table"][:, :n_blk].long()

    def rows(codes, scale):     # [b, h_kv, n_blk * 64, d]
        x = codes.view(torch.int8)[table].view(codes.dtype).float() * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(b, h_kv, n_blk * BLOCK, d)

    i = torch.arange(s["total"], device=DEV)
    r = torch.bucketize(i, cu[1:], right=True)
    t = i - cu[r]
    Q = s["max_q"]
    q = torch.zeros((b, Q, c["h_q"], d), device=DEV)
    q[r, t] = s["q"].float()
    q = q.view(b, Q, h_kv, g, d).permute(0, 2, 3, 1, 4).reshape(b, h_kv, g * Q, d)
    x = torch.matmul(q, rows(s["k_cache"], s["k_scale"]).transpose(2, 3)).view(b, h_kv, g, Q, -1)
    x *= 1.0 / math.sqrt(d)
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    j = torch.arange(n_blk * BLOCK, device=DEV)
    pos = (kv - (cu[1:] - cu[:-1]))[:, None] + torch.arange(Q, device=DEV)[None]      # [b, Q]
    if c["alibi"]:
        far = (pos[:, :, None] - j).abs().float()[:, None, None]
        x = x - s["slopes"].view(1, h_kv, g, 1, 1) * far
    seen = (j[None, None] < kv[:, None, None]).expand(b, Q, -1)
    if c["causal"]:
        reach = pos + 1
        if s["prefix"] is not None:
            reach = torch.maximum(reach, s["prefix"].long()[:, None])
        seen = seen & (j[None, None] < reach[:, :, None])
    if s["docs"] is not None:
        bounds = torch.zeros((b, Q, 2), dtype=torch.int64, device=DEV)
        bounds[r, t] = s["docs"].long()
        seen = seen & (j >= bounds[:, :, :1]) & (j < bounds[:, :, 1:])
    seen = seen[:, None, None]
    x = torch.where(seen, x, torch.full((), -math.inf, device=DEV))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    del x
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, h_kv, g * Q, -1), rows(s["v_cache"], s["v_scale"])).view(b, h_kv, g, Q, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (torch.log(total) + top).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, Q, c["h_q"], d)[r, t]
    lse = lse.permute(0, 3, 1, 2).reshape(b, Q, c["h_q"])[r, t]
    return o.to(torch.bfloat16), lse


# --------------------------------------------------------------------------- one pass
def run(s):
    c = s["c"]
    if own:
        import sparse_mla_decoding_b200 as smla
        if c["op"] == "table":
            slots, cu, lens, left = smla.extend_block_table(s["block_table"], s["cache_seqlens"], s["new_lens"],
                                                            s["free_blocks"], s["num_free"], s["max_new_tokens"])
            return slots, cu, lens, left, s["block_table"]
        if c["op"] == "write":
            smla.quantize_kv_blocks(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                    s["block_table"], s["cache_seqlens"], s["new_seqlens"], s["cu"])
            return s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]
        return smla.gqa_attention_with_kvcache(
            s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["cache_seqlens"],
            cu_seqlens_q=s["cu"], max_seqlen_q=s["max_q"], causal=c["causal"], softcap=c["softcap"],
            alibi_slopes=s["slopes"], prefix_lens=s["prefix"], doc_bounds=s["docs"])
    if c["op"] == "table":
        return _table_plain(s)
    if c["op"] == "write":
        return _write_plain(s)
    return _attend_plain(s)


# --------------------------------------------------------------------------- 64 bits
def _exact_attend(c, s):
    lo, hi = _visible(c)
    q_lens, kv_lens = _lens(c)
    g, d = c["h_q"] // c["h_kv"], c["d"]
    kc, vc = s["k_cache"].view(torch.int8), s["v_cache"].view(torch.int8)
    o = torch.zeros((s["total"], c["h_q"], d), dtype=torch.float64, device=DEV)
    lse = torch.full((s["total"], c["h_q"]), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for r in range(c["batch"]):
        n, L = int(q_lens[r]), int(kv_lens[r])
        blocks = s["block_table"][r, :-(-L // BLOCK)].long()
        first, end = torch.from_numpy(lo[r]).to(DEV), torch.from_numpy(hi[r]).to(DEV)
        j = torch.arange(L, device=DEV)
        hide = (j[None] < first[:, None]) | (j[None] >= end[:, None])
        pos = torch.arange(L - n, L, device=DEV)
        for h in range(c["h_kv"]):
            ks, vs = (x[blocks, h].double()[:, None, None] for x in (s["k_scale"], s["v_scale"]))
            k = (kc[blocks, h].view(s["k_cache"].dtype).double() * ks).reshape(-1, d)[:L]
            v = (vc[blocks, h].view(s["v_cache"].dtype).double() * vs).reshape(-1, d)[:L]
            for e in range(h * g, (h + 1) * g):
                x = s["q"][at:at + n, e].double() @ k.T / math.sqrt(d)
                if c["softcap"]:
                    x = torch.tanh(x / c["softcap"]) * c["softcap"]
                if c["alibi"]:
                    x -= s["slopes"][e].double() * (pos[:, None] - j[None]).abs()
                x.masked_fill_(hide, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[at:at + n, e] = z
                o[at:at + n, e] = torch.nan_to_num(torch.exp(x - z[:, None])) @ v
        at += n
    return o, lse


def exact(c, seed):
    if c["op"] == "table":
        return None        # whole numbers
    s = prepare(c, seed)
    if c["op"] == "attend":
        return _exact_attend(c, s)
    # The writer's scales; its codes are held to the plain form's (float8 by value, int8 to the last one).
    q, kv = _lens(c)
    out = []
    for x, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        scale = scale.double()
        table, at = s["block_table"].cpu().numpy(), 0
        most = x.double().abs().amax(-1)
        for r in range(c["batch"]):
            n, old = int(q[r]), int(kv[r] - q[r])
            for j in range(old // BLOCK, -(-(old + n) // BLOCK) if n else 0):
                a, e = max(0, j * BLOCK - old), min(n, (j + 1) * BLOCK - old)
                top = most[at + a:at + e].amax(0)
                # two bf16 ratios differ by 2^-8 at least: the small step keeps log2's last bit out of the ceiling
                k = torch.ceil(torch.log2(top / (448.0 if c["cache"] == "e4m3" else 127.0)) - 1e-9)
                new = torch.where(top > 0, torch.exp2(k), torch.zeros_like(top))
                blk = int(table[r, j])
                scale[blk] = torch.maximum(new, scale[blk]) if j * BLOCK < old else new
            at += n
        out += [None, scale]
    return tuple(out)
