"""The paged operators' definitions in float64 numpy, for the tests: written from
the formulas, one request and one head at a time."""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 64


def extend_block_table(table, lens, new, free, num_free, max_new):
    """(table, slots, cu, lens out, left) by the rule of the block-table entry point."""
    table = table.copy()
    slots = np.full(max_new, -1, np.int64)
    cu = np.zeros(len(lens) + 1, np.int64)
    out = lens.copy()
    asked = taken = 0
    for r in range(len(lens)):
        n = max(int(new[r]), 0)
        cu[r + 1] = cu[r] + n
        before, after = -(-int(lens[r]) // BLOCK), -(-(int(lens[r]) + n) // BLOCK)
        need = after - before
        if after > table.shape[1]:
            continue                              # no room in its row: asks for nothing
        first = asked
        asked += need
        if (need and asked > num_free) or cu[r + 1] > max_new:
            continue
        for i in range(need):
            table[r, before + i] = free[num_free - 1 - first - i]
        taken += need
        out[r] = lens[r] + n
        for t in range(n):
            p = int(lens[r]) + t
            slots[cu[r] + t] = int(table[r, p // BLOCK]) * BLOCK + p % BLOCK
    return table, slots, cu.astype(np.int32), out.astype(np.int32), num_free - taken


def visible(n, length, t, causal, prefix=0, doc=None):
    lo, hi = 0, length
    if causal:
        hi = min(hi, max(length - n + t + 1, prefix))
    if doc is not None:
        lo, hi = max(lo, int(doc[0])), min(hi, int(doc[1]))
    return lo, max(lo, hi)


def attention(q, k, v, table, lens, cu, scale=None, causal=True, softcap=0.0, slopes=None, prefix=None, docs=None,
              v_scale=None):
    """(o, lse, o tolerance, lse tolerance), float64, of q [total, h_q, d] over k, v
    [num_blocks, h_kv, 64, d] (codes times scales, float64; v_scale [num_blocks, h_kv]).

    The tolerances count the kernel's roundings.  The output: half a bf16 step, 2^-8 of
    |o| and of what else it is off by.  P to f16: 2^-11 of sum p|v|.  A score: its fp32
    accumulation over d / 16 <= 8 matrix steps, 8 * 2^-23 of sum |q k|, and a few more
    roundings of the scaled, capped and biased score and of exp2, within 2^-20 (1 +
    |parts|): together 2^-19 of the score's parts, which moves lse by as much and o by
    twice that of sum p|v|.

    Below 2^-14 f16's steps are 2^-24, so such a P is off by up to 2^-25 absolutely
    instead.  P_j = 2^(x_j - M) s_j with the value scale s_j, and the output is sum_j P_j
    c_j 2^M / sum_j 2^x_j with the codes c_j.  M is the largest x_i + log2 s_i at the last
    rescaling, so 2^M / sum_j 2^x_j <= max_i w_i s_i with the weights w_i, and these
    errors together are at most 2^-25 sum_j |c_j| max_i w_i s_i."""
    q = np.asarray(q, np.float64)
    total, h_q, d = q.shape
    g = h_q // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o = np.zeros((total, h_q, d))
    lse = np.full((total, h_q), -np.inf)
    tol = np.zeros((total, h_q, d))
    tol_lse = np.zeros((total, h_q))
    for r in range(len(lens)):
        n, L = int(cu[r + 1] - cu[r]), int(lens[r])
        if L == 0 or n == 0:
            continue
        blocks = table[r, :-(-L // BLOCK)]
        gone = (blocks < 0) | (blocks >= k.shape[0])
        at = np.where(gone, 0, blocks)
        there = np.repeat(~gone, BLOCK)[:L]
        for h in range(h_q):
            K = k[at, h // g].reshape(-1, d)[:L]
            V = v[at, h // g].reshape(-1, d)[:L]
            s = np.repeat(v_scale[at, h // g], BLOCK)[:L]
            C = np.abs(V) / np.where(s > 0, s, 1)[:, None]
            for t in range(n):
                i, p = int(cu[r]) + t, L - n + t
                lo, hi = visible(n, L, t, causal, 0 if prefix is None else int(prefix[r]),
                                 None if docs is None else docs[i])
                j = np.arange(lo, hi)[there[lo:hi]]
                if len(j) == 0:
                    continue
                x = K[j] @ q[i, h] * scale
                parts = np.abs(K[j]) @ np.abs(q[i, h]) * scale
                if softcap > 0:
                    x = softcap * np.tanh(x / softcap)
                    parts = parts + softcap
                if slopes is not None:
                    x = x - slopes[h] * np.abs(p - j)
                    parts = parts + slopes[h] * np.abs(p - j)
                m = x.max()
                e = np.exp(x - m)
                w = e / e.sum()
                lse[i, h] = m + np.log(e.sum())
                o[i, h] = w @ V[j]
                near = w > 1e-12                      # parts of scores that carry no weight move nothing
                delta = 2.0 ** -19 * (1 + parts[near].max() + abs(lse[i, h]))
                tol_lse[i, h] = delta
                off = (2.0 ** -11 + 2 * delta) * (w @ np.abs(V[j])) + 2.0 ** -25 * C[j].sum(0) * (w * s[j]).max()
                tol[i, h] = 2.0 ** -8 * (np.abs(o[i, h]) + off) + off
    return o, lse, tol, tol_lse


def compare(o, lse, ref, rows=None):
    o_ref, l_ref, tol, tol_lse = ref
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    if rows is not None:
        o, lse, o_ref, l_ref, tol, tol_lse = (a[rows] for a in (o, lse, o_ref, l_ref, tol, tol_lse))
    dead = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(lse), dead), "-inf lse in other places"
    assert (o[dead] == 0).all(), "o must be 0 where nothing is seen"
    assert np.isfinite(o).all()
    over = np.abs(o - o_ref) - tol
    assert over.max(initial=-1) <= 0, f"o is {over.max():.3e} beyond its tolerance"
    off = np.abs(lse[~dead] - l_ref[~dead]) - tol_lse[~dead]
    assert off.max(initial=-1) <= 0, f"lse is {off.max():.3e} beyond its tolerance"


CACHE_TYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def make_cache(num_blocks, h_kv, d, kind, seed, spread=True):
    """(codes, scales, codes * scales in float64) of one side of a cache, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(num_blocks, h_kv, BLOCK, d, generator=g)
    if kind == "e4m3":
        codes = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        codes = (x * 40).round().clamp(-127, 127).to(torch.int8)
    scale = torch.rand(num_blocks, h_kv, generator=g) * 0.015 + 0.005
    if spread:                                       # blocks far apart in size
        scale = scale * torch.exp2(torch.randint(-3, 3, (num_blocks, h_kv), generator=g).float())
    return codes, scale, codes.double().numpy() * scale.double().numpy()[:, :, None, None]


def make_table(lens, seed, extra=2, spare=3):
    rng = np.random.default_rng(seed)
    need = [-(-int(x) // BLOCK) for x in lens]
    perm = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lens), max(need + [1]) + extra), 1 << 29, np.int32)   # unused entries point nowhere
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, sum(need) + spare
