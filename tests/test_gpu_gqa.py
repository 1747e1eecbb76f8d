"""Grouped-query attention over the block-scaled 8-bit cache on the GPU against the
definition in float64: head groups, lengths around the blocks' edges, one and many
new tokens, capped and biased scores, masks that leave rows empty, split schedules."""
import numpy as np
import pytest
import torch

import paged_util as U

pytestmark = pytest.mark.gpu


def build(q_lens, lens, h_q, h_kv, d, kind, seed, poison=True):
    """Inputs on the host; rows behind a request's length and blocks of no request hold NaN (e4m3)."""
    lens, q_lens = np.asarray(lens, np.int32), np.asarray(q_lens, np.int32)
    table, blocks = U.make_table(lens, seed)
    kc, ks, k = U.make_cache(blocks, h_kv, d, kind, seed + 1)
    vc, vs, v = U.make_cache(blocks, h_kv, d, kind, seed + 2)
    if poison:
        dead = np.ones((blocks, U.BLOCK), bool)
        for r, n in enumerate(lens):
            for b in range(-(-int(n) // U.BLOCK)):
                dead[table[r, b], :min(U.BLOCK, int(n) - b * U.BLOCK)] = False
        mask = torch.from_numpy(dead)[:, None, :, None].expand(kc.shape)
        for c in (kc, vc):
            c.view(torch.int8)[mask] = 127      # NaN in e4m3
    g = torch.Generator().manual_seed(seed + 3)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = (torch.randn(int(cu[-1]), h_q, d, generator=g) * 1.5).to(torch.bfloat16)
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=lens, cu=cu, k=k, v=v)


LONG = 1 << 20      # more than any call's tokens: picks the kernel for long prompts


def call(x, four_d=None, **kw):
    """Unless a test says which, the kernel for long prompts from 33 rows of a request on."""
    rows = int(np.diff(x["cu"]).max()) * (x["q"].shape[1] // x["kc"].shape[1])
    kw.setdefault("max_seqlen_q", LONG if rows > 32 else 1)
    import sparse_mla_decoding_b200 as smla
    dev = {n: x[n].cuda() if isinstance(x[n], torch.Tensor) else torch.from_numpy(x[n]).cuda()
           for n in ("q", "kc", "vc", "ks", "vs", "table", "lens", "cu")}
    gpu = {n: torch.from_numpy(np.asarray(a)).cuda() if isinstance(a, np.ndarray) else a for n, a in kw.items()}
    ws = smla.new_gqa_workspace(dev["kc"].shape[3])
    q, cu = (dev["q"], dev["cu"]) if four_d is None else (dev["q"].view(four_d), None)
    o, lse = smla.gqa_attention_with_kvcache(q, dev["kc"], dev["vc"], dev["ks"], dev["vs"], dev["table"], dev["lens"],
                                             cu_seqlens_q=cu, workspace=ws, **gpu)
    torch.cuda.synchronize()
    return o, lse, smla.get_device_status(ws)


def reference(x, **kw):
    names = {"alibi_slopes": "slopes", "prefix_lens": "prefix", "doc_bounds": "docs", "softmax_scale": "scale"}
    kw = {names.get(n, n): a for n, a in kw.items() if n != "max_seqlen_q"}
    return U.attention(x["q"].double().numpy(), x["k"], x["v"], x["table"], x["lens"], x["cu"],
                       v_scale=x["vs"].double().numpy(), **kw)


def check(x, **kw):
    """By both kernels, and by the one that the sizes pick."""
    ref = reference(x, **kw)
    for hint in [None, 1, LONG] if "max_seqlen_q" not in kw else [kw["max_seqlen_q"]]:
        o, lse, (status, raw) = call(x, **{**kw, "max_seqlen_q": hint})
        assert status == 0, f"flags {raw:#x}"
        U.compare(o, lse, ref)
    return o, lse


KINDS = ["e4m3", "int8"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h_q,h_kv", [(8, 8), (8, 1), (14, 2), (5, 5), (32, 1)])
def test_single_tokens(h_q, h_kv, d, kind):
    """Lengths of one token, around a block's and a tile's edge, and over several blocks."""
    x = build([1] * 8, [1, 2, 63, 64, 65, 129, 500, 17], h_q, h_kv, d, kind, 100 + d + h_q)
    check(x)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_several_tokens_and_empty_requests(d, kind):
    """Requests without new tokens, without a cache, with more new tokens than one row tile holds."""
    x = build([3, 0, 1, 7, 0, 70, 2], [300, 5, 1, 7, 0, 200, 64], 12, 4, d, kind, 200 + d)
    check(x)


@pytest.mark.parametrize("d", [64, 128])
def test_more_new_tokens_than_cache(d):
    """Tokens before the start of the cache see nothing."""
    x = build([5, 4], [2, 0], 4, 2, d, "e4m3", 250 + d)
    o, lse = check(x)
    assert torch.isinf(lse[:3]).all() and torch.isinf(lse[5:]).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("mods", ["cap", "cap_small", "alibi", "cap+alibi", "full", "full+alibi"])
def test_scores(mods, kind):
    x = build([1, 4, 40, 1], [400, 129, 130, 3], 16, 2, 128, kind, 300)
    kw = {}
    if "cap" in mods:
        kw["softcap"] = 0.8 if "small" in mods else 30.0
    if "alibi" in mods:
        kw["alibi_slopes"] = np.exp2(-np.arange(16) / 2).astype(np.float32)
    if "full" in mods:
        kw["causal"] = False
    check(x, **kw)


@pytest.mark.parametrize("d", [64, 128])
def test_prefix(d):
    """A prefix longer than the causal reach, shorter, zero, and past the end of the cache."""
    x = build([20, 20, 1, 33], [20, 150, 100, 70], 8, 4, d, "int8", 400 + d)
    check(x, prefix_lens=np.array([9, 140, 0, 5000], np.int32))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_documents(d, causal):
    """Documents that start inside a block, that hold one token, that end before their token and that are empty."""
    x = build([1, 6, 50, 1], [700, 70, 300, 40], 8, 2, d, "e4m3", 500 + d)
    docs = [(650, 700)] + [(64, 65), (65, 70), (0, 64), (66, 66), (30, 1000), (-5, 3)]
    docs += [(200, 290)] * 30 + [(290, 300)] * 20 + [(20, 10)]
    o, lse = check(x, doc_bounds=np.array(docs, np.int32), causal=causal)
    assert torch.isinf(lse[-1]).all() and (o[-1] == 0).all()


@pytest.mark.parametrize("causal", [True, False])
def test_documents_that_end_far_below_zero(causal):
    lo, hi = -(1 << 31), (1 << 31) - 1
    x = build([6, 50], [300, 310], 8, 2, 64, "int8", 2000)
    docs = [(0, 300), (0, lo), (hi, lo), (lo, lo), (hi, hi), (lo, hi)] + [(0, 310), (0, lo), (hi, lo), (7, -5), (lo, hi)] * 10
    check(x, doc_bounds=np.array(docs, np.int32), causal=causal)


def test_prefix_and_documents_and_bias_together():
    x = build([40, 3], [200, 90], 6, 2, 128, "e4m3", 550)
    docs = np.array([(0, 180)] * 20 + [(180, 200)] * 20 + [(10, 90)] * 3, np.int32)
    check(x, doc_bounds=docs, prefix_lens=np.array([100, 0], np.int32), softcap=20.0,
          alibi_slopes=np.full(6, 0.05, np.float32), softmax_scale=0.11)


@pytest.mark.parametrize("kind", KINDS)
def test_split_over_many_warps(kind):
    """One long request: its blocks are spread over many warps and merged."""
    x = build([1, 2], [20011, 1500], 8, 2, 128, kind, 600)
    check(x)


def test_many_short_requests():
    """More requests than a CTA has threads, each shorter than a block or two."""
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 100, 700)
    x = build(np.minimum(1, lens), lens, 4, 2, 64, "int8", 700)
    check(x)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [1, 2])
def test_ragged_batches_cut_everywhere(tokens, d):
    """Ranges of CTAs and warps that begin and end at all places of a unit."""
    rng = np.random.default_rng(d + tokens)
    lens = np.concatenate([rng.integers(tokens, 200, 30), rng.integers(200, 3000, 12)])
    rng.shuffle(lens)
    x = build([tokens] * len(lens), lens, 12, 2, d, "int8", 750 + d + tokens)
    check(x)


def test_four_dimensional_queries_equal_packed_ones():
    x = build([3] * 5, [3, 64, 100, 259, 30], 8, 4, 128, "e4m3", 800)
    o, lse, _ = call(x)
    o4, lse4, _ = call(x, four_d=(5, 3, 8, 128))
    assert torch.equal(o.view(5, 3, 8, 128), o4) and torch.equal(lse.view(5, 3, 8), lse4)


@pytest.mark.parametrize("hint", [1, 4, 100000])
def test_hint_changes_nothing_that_is_computed(hint):
    x = build([1, 30, 2], [100, 90, 300], 8, 2, 128, "e4m3", 850)
    check(x, max_seqlen_q=hint)


@pytest.mark.parametrize("hint", [1 << 31, 1 << 40])
def test_hints_of_any_size(hint):
    x = build([1, 30], [100, 90], 8, 2, 128, "e4m3", 2010)
    check(x, max_seqlen_q=hint)


@pytest.mark.parametrize("n", [1, 40])
def test_zero_scales_and_large_spreads(n):
    """Blocks of zero keys or values beside ordinary ones, and scales far apart."""
    x = build([n], [400], 8, 2, 128, "int8", 900, poison=False)
    blocks = x["table"][0, :7]
    x["vs"][blocks[1]] = 0
    x["vs"][blocks[3]] *= 2.0 ** 30
    x["vs"][blocks[4]] *= 2.0 ** -25
    x["ks"][blocks[2]] = 0
    for codes, scale, name in (("kc", "ks", "k"), ("vc", "vs", "v")):
        x[name] = x[codes].double().numpy() * x[scale].double().numpy()[:, :, None, None]
    check(x)


@pytest.mark.parametrize("size", [2.0 ** -112, 2.0 ** -100, 2.0 ** 100])
@pytest.mark.parametrize("n", [1, 40])
def test_zero_value_scales_before_far_ones(n, size):
    """The first blocks hold zeros (scale 0), the others values far from 1.  bf16's steps below
    2^-126 are 2^-133, so the rounding of o there is off by up to 2^-134 whatever its size."""
    x = build([n], [900], 8, 2, 64, "int8", 2020, poison=False)
    blocks = x["table"][0, :15]
    x["vs"][blocks] *= size
    x["vs"][blocks[[0, 1, 9]]] = 0
    x["vc"][blocks[[0, 1, 9]]] = 0
    x["v"] = x["vc"].double().numpy() * x["vs"].double().numpy()[:, :, None, None]
    o_ref, lse_ref, tol, tol_lse = reference(x)
    for hint in (None, 1, LONG):
        o, lse, (status, _) = call(x, max_seqlen_q=hint)
        assert status == 0
        U.compare(o, lse, (o_ref, lse_ref, tol + 2.0 ** -134, tol_lse))


@pytest.mark.parametrize("d", [64, 128])
def test_many_blocks_of_zeros_before_far_values(d):
    """More than 32 blocks whose value scale is 0 in one CTA's or warp's run of blocks."""
    x = build([9] * 10, [2500, 2400] + [60] * 8, 32, 8, d, "int8", 2030 + d, poison=False)
    zeros = x["table"][:2, :35]
    x["vs"] *= 2.0 ** -100
    x["vs"][zeros] = 0
    x["vc"][zeros] = 0
    x["v"] = x["vc"].double().numpy() * x["vs"].double().numpy()[:, :, None, None]
    check(x)


@pytest.mark.parametrize("d", [64, 128])
def test_sums_over_values_of_zero(d):
    """All value scales 0: o is 0, and lse as precise as ever, of rows that see one key each."""
    x = build([70], [140], 32, 1, d, "int8", 2050 + d, poison=False)
    x["vs"].zero_()
    x["v"] = np.zeros_like(x["v"])
    at = np.arange(70)
    o, lse = check(x, softmax_scale=0.003, doc_bounds=np.stack([at, at + 1], 1).astype(np.int32))
    assert (o == 0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,d", [(1, 64), (1, 128), (40, 64), (40, 128)])
def test_values_of_a_zero_scale(n, d, kind):
    """A block whose codes stand for zeros takes all but e^-20 of the weight: o is what the others
    give.  A NaN among them is a NaN for the tokens that see it (e4m3)."""
    x = build([n], [300], 8, 2, d, kind, 2070 + d, poison=False)
    block = x["table"][0, 0]
    u = torch.sign(torch.randn(d, generator=torch.Generator().manual_seed(d)))
    x["q"][:] = u
    x["kc"][block] = u.to(x["kc"].dtype)
    x["ks"] *= 0.02
    x["ks"][block] = 20.0 / d
    x["vs"][block] = 0
    x["k"], x["v"] = (x[c].double().numpy() * x[s].double().numpy()[:, :, None, None]
                      for c, s in (("kc", "ks"), ("vc", "vs")))
    check(x, softmax_scale=1.0)
    if kind == "e4m3":
        x["vc"].view(torch.int8)[block, 0, 5, 3] = 127
        ref = reference({**x, "v": np.nan_to_num(x["v"])}, softmax_scale=1.0)
        for hint in (1, LONG):
            o, lse, _ = call(x, softmax_scale=1.0, max_seqlen_q=hint)
            assert torch.isnan(o[:, :4, 3]).all() and torch.isfinite(lse).all()
            o[:, :4, 3] = torch.from_numpy(ref[0]).cuda()[:, :4, 3].to(o.dtype)
            U.compare(o, lse, ref)


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_far_query_sizes(size):
    """Queries far outside f16's range: scores of ordinary size come from the softmax scale."""
    x = build([2], [90], 4, 2, 64, "e4m3", 950)
    x["q"] = (x["q"].double() * size).to(torch.bfloat16)
    check(x, softmax_scale=float(0.125 / size))


@pytest.mark.parametrize("hint", [1, LONG])
@pytest.mark.parametrize("mods", ["", "cap", "slopes", "alone"])
def test_a_nan_key_reaches_every_row_that_sees_it(mods, hint):
    """At each place among eight neighbours, and as the only key that a row sees; other rows and heads are as ever."""
    kw = {"max_seqlen_q": hint}
    if mods == "cap":
        kw["softcap"] = 30.0
    if mods == "slopes":
        kw["alibi_slopes"] = np.full(8, 0.05, np.float32)
    for at in range(176, 184):
        x = build([40, 1], [200, 190], 8, 2, 128 if at % 2 else 64, "e4m3", 1900 + at)
        if mods == "alone":
            kw["doc_bounds"] = np.array([(0, 200)] * 39 + [(at, at + 1)] + [(at, at + 1)], np.int32)
        for r in range(2):
            x["kc"].view(torch.int8)[x["table"][r, at // 64], 0, at % 64, 11] = 127
        o, lse, (status, _) = call(x, **kw)
        assert status == 0
        sees = np.zeros((41, 8), bool)
        sees[at - 160:, :4] = True                    # tokens at positions 160 .. 199, and the other request's
        hit = torch.from_numpy(sees)
        assert torch.isnan(o.cpu()[hit]).all() and torch.isnan(lse.cpu()[hit]).all()
        U.compare(o, lse, reference(x, **kw), rows=~sees)


@pytest.mark.parametrize("hint", [1, LONG])
@pytest.mark.parametrize("length", [50, 190])
def test_a_token_that_sees_nothing_beside_nan_values(length, hint):
    x = build([2, 2], [length, length + 1], 8, 2, 128, "e4m3", 1950)
    x["vc"].view(torch.int8)[x["table"][:, 0], :, 3] = 127
    docs = np.array([(5, 5), (0, 1000)] * 2, np.int32)
    o, lse, (status, _) = call(x, doc_bounds=docs, max_seqlen_q=hint)
    assert status == 0
    assert (o[::2] == 0).all() and torch.isneginf(lse[::2]).all()
    assert torch.isnan(o[1::2]).all() and torch.isfinite(lse[1::2]).all()


@pytest.mark.parametrize("mods", ["cap", "cap+slopes", "slopes", ""])
@pytest.mark.parametrize("n", [1, 40])
def test_zero_scores_under_extreme_scales(n, mods):
    """All scores are 0 whatever they are multiplied by: o is the mean of the values."""
    x = build([n], [150], 8, 2, 64, "int8", 1960, poison=False)
    x["kc"].zero_()
    x["ks"].fill_(1.0)
    x["k"] = np.zeros_like(x["k"])
    kw = {"alibi_slopes": np.full(8, 0.01, np.float32)} if "slopes" in mods else {}
    for scale, cap in [(1e6, 1.0), (1e38, 1.0), (1e38, 2.0 ** -60), (1e30, 2.0 ** 60)]:
        check(x, softmax_scale=scale, **({"softcap": cap} if "cap" in mods else {}), **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 40])
def test_small_probabilities_beside_a_large_one_reach_the_output(n, kind):
    """Each block's first key has e^18 = 2^25.97 times the weight of each other, and value 0:
    o = w / (1 + w) of the others' weight w.  P is at least 2^7 at the running maximum, so the
    others' are 2^-18.97 or more, where f16 is off by at most 2^-25, 2^-6.03 of it; with the
    half step of o 2^-8 and 2^-10 for all else."""
    x = build([n], [290], 4, 1, 64, kind, 1970, poison=False)
    for c in ("kc", "vc"):
        x[c].copy_(torch.zeros(x[c].shape).to(x[c].dtype))
    x["kc"][:, :, 0, 0] = 18.0 if kind == "e4m3" else 18
    x["vc"][:, :, 1:] = 1.0 if kind == "e4m3" else 1
    x["ks"].fill_(1.0)
    x["vs"].fill_(1.0)
    x["k"], x["v"] = x["kc"].double().numpy(), x["vc"].double().numpy()
    x["q"].zero_()
    x["q"][:, :, 0] = 1.0
    ref = U.attention(x["q"].double().numpy(), x["k"], x["v"], x["table"], x["lens"], x["cu"], scale=1.0,
                      v_scale=x["vs"].double().numpy())[0]
    for hint in (1, LONG):
        o = call(x, softmax_scale=1.0, max_seqlen_q=hint)[0].double().cpu().numpy()
        assert (np.abs(o - ref) <= (2.0 ** -6.03 + 2.0 ** -8 + 2.0 ** -10) * ref).all()


def test_strided_queries_scales_and_blocks():
    """Query rows inside a fused projection; keys and values in one allocation."""
    import sparse_mla_decoding_b200 as smla
    x = build([2, 1], [100, 257], 8, 2, 128, "e4m3", 1000)
    nb = x["kc"].shape[0]
    both = torch.zeros(nb, 2, 2, 64, 128, dtype=torch.int8, device="cuda")
    both[:, 0], both[:, 1] = x["kc"].view(torch.int8).cuda(), x["vc"].view(torch.int8).cuda()
    both = both.view(torch.float8_e4m3fn)
    scales = torch.stack([x["ks"], x["vs"]], 1).cuda()
    fused = torch.full((3, 12, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:10] = x["q"].cuda()
    args = [torch.from_numpy(x[n]).cuda() for n in ("table", "lens")]
    o, lse = smla.gqa_attention_with_kvcache(fused[:, 2:10], both[:, 0], both[:, 1], scales[:, 0], scales[:, 1], *args,
                                             cu_seqlens_q=torch.from_numpy(x["cu"]).cuda(), check_device_status=True)
    U.compare(o, lse, reference(x))


@pytest.mark.parametrize("shape", [(1, 1), (2, 1), (1, 3), (2, 3)])
@pytest.mark.parametrize("h_q", [1, 4])
def test_odd_query_strides_and_alignments(shape, h_q):
    """Queries that 16-byte loads cannot read as they are, and strides of lone dimensions."""
    import sparse_mla_decoding_b200 as smla
    b, s_q = shape
    x = build([s_q] * b, [70] * b, h_q, 1, 64, "int8", 1050 + h_q)
    q = x["q"].view(b, s_q, h_q, 64).cuda()
    n = q.numel()
    odd = torch.empty(n + 1, dtype=torch.bfloat16, device="cuda")[1:].view(q.shape)
    odd.copy_(q)
    wide = torch.empty(b, s_q, h_q, 67, dtype=torch.bfloat16, device="cuda")[..., :64]
    wide.copy_(q)
    turned = torch.empty(s_q, b, h_q, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    turned.copy_(q)
    lone = q.as_strided(q.shape, tuple(st if sz > 1 else 5 for sz, st in zip(q.shape, q.stride())))
    apart = torch.empty(b, s_q + 2, h_q, 64, dtype=torch.bfloat16, device="cuda")[:, :s_q]
    apart.copy_(q)
    args = [x[k].cuda() for k in ("kc", "vc", "ks", "vs")] + [torch.from_numpy(x[k]).cuda() for k in ("table", "lens")]
    ref = reference(x)
    for t in (q, odd, wide, turned, lone, apart):
        o, lse = smla.gqa_attention_with_kvcache(t, *args, check_device_status=True)
        assert o.is_contiguous() and o.shape == q.shape
        U.compare(o.view(-1, h_q, 64), lse.view(-1, h_q), ref)


@pytest.mark.parametrize("n", [1, 40])
def test_rows_behind_the_last_request_are_left(n):
    import sparse_mla_decoding_b200 as smla
    x = build([n, n], [100, 70], 8, 2, 128, "e4m3", 1100)
    q = torch.cat([x["q"], torch.full((7, 8, 128), float("nan"), dtype=torch.bfloat16)]).cuda()
    o = torch.full((2 * n + 7, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2 * n + 7, 8), 5.0, device="cuda")
    smla.gqa_attention_with_kvcache(q, x["kc"].cuda(), x["vc"].cuda(), x["ks"].cuda(), x["vs"].cuda(),
                                    *(torch.from_numpy(x[k]).cuda() for k in ("table", "lens", "cu")), out=(o, lse),
                                    max_seqlen_q=1 if n == 1 else LONG)
    U.compare(o[:2 * n], lse[:2 * n], reference(x))
    assert (o[2 * n:] == 3).all() and (lse[2 * n:] == 5).all()


@pytest.mark.parametrize("n", [1, 40])
def test_bad_blocks_are_skipped_and_flagged(n):
    x = build([n], [300], 8, 2, 128, "e4m3", 1200)
    x["table"][0, 1] = -7
    x["table"][0, 3] = x["kc"].shape[0]
    o, lse, (status, raw) = call(x)
    assert status == 1 and raw == 2
    U.compare(o, lse, reference(x))


@pytest.mark.parametrize("n", [1, 40])
def test_length_past_the_table_is_flagged(n):
    x = build([n], [128], 4, 2, 64, "int8", 1250)
    x["table"] = np.ascontiguousarray(x["table"][:, :2])
    x["lens"] = np.array([1000], np.int32)
    o, lse, (status, raw) = call(x, causal=False)
    assert status == 1 and raw == 2
    x["table"] = np.concatenate([x["table"], np.full((1, 20), -1, np.int32)], 1)
    U.compare(o, lse, reference(x, causal=False))


def test_bad_offsets_are_flagged_and_leave_the_others():
    x = build([2, 3, 2], [100, 80, 90], 4, 2, 64, "e4m3", 1300)
    ref = reference(x)
    x["cu"] = np.array([0, 2, 1, 7], np.int32)      # request 1 runs backwards, request 2 claims rows 1 .. 6
    o, lse, (status, raw) = call(x)
    assert status == 1 and raw & 4
    U.compare(o[:1], lse[:1], [a[:1] for a in ref])


def test_bad_offsets_of_long_requests_are_flagged():
    """More than the decode kernel's rows: the request that runs past the end is left out."""
    x = build([40, 50], [100, 80], 4, 2, 64, "e4m3", 1320)
    ref = reference(x)
    x["cu"] = np.array([0, 40, 91], np.int32)
    o, lse, (status, raw) = call(x)
    assert status == 1 and raw & 4
    U.compare(o[:40], lse[:40], [a[:40] for a in ref])


@pytest.mark.parametrize("n", [1, 40])
def test_blocks_past_two_gigabytes(n):
    """A cache of more than 2^31 bytes a side, with the request's blocks at its end."""
    import sparse_mla_decoding_b200 as smla
    x = build([n], [200], 16, 8, 128, "int8", 1350, poison=False)
    nb, used = 33000, x["kc"].shape[0]
    big = {}
    for c, s in (("kc", "ks"), ("vc", "vs")):
        big[c] = torch.empty(nb, 8, 64, 128, dtype=torch.int8, device="cuda")
        big[s] = torch.empty(nb, 8, device="cuda")
        big[c][nb - used:] = x[c].cuda()
        big[s][nb - used:] = x[s].cuda()
    table = torch.from_numpy(x["table"]).cuda()
    table[:, :4] += nb - used
    args = [torch.from_numpy(x[k]).cuda() for k in ("lens", "cu")]
    o, lse = smla.gqa_attention_with_kvcache(x["q"].cuda(), big["kc"], big["vc"], big["ks"], big["vs"], table, args[0],
                                             cu_seqlens_q=args[1], max_seqlen_q=1 if n == 1 else LONG,
                                             check_device_status=True)
    U.compare(o, lse, reference(x))
    k = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    before = big["kc"][nb - used:].clone()
    smla.quantize_kv_blocks(k, k, big["kc"], big["vc"], big["ks"], big["vs"], table, args[0] - 3, args[0], cu,
                            check_device_status=True)
    last = int(table[0, 3])
    rows = big["kc"][last, :, 5:8].float() * big["ks"][last][:, None, None]
    assert (rows - k.float().transpose(0, 1)).abs().max() <= big["ks"][last].max() / 2
    before[last - (nb - used)] = big["kc"][last]
    assert torch.equal(before, big["kc"][nb - used:])


@pytest.mark.parametrize("kind,d", [("e4m3", 128), ("int8", 64)])
@pytest.mark.parametrize("mods", ["", "docs", "cap prefix slopes"])
def test_rows_shared_by_several_ctas(mods, kind, d):
    """Few row tiles over long lengths: parts that some or all rows do not see, a request too
    short to be shared, lengths that end inside a block, rows that end inside a tile."""
    q_lens, lens = [150, 3, 20, 140], [4000, 90, 2777, 140]
    x = build(q_lens, lens, 8, 2, d, kind, 1700 + d)
    kw = {}
    if "docs" in mods:
        rng = np.random.default_rng(d)
        total = sum(q_lens)
        lo = rng.integers(0, 2600, total)
        docs = np.stack([lo, lo + rng.integers(0, 900, total)], 1).astype(np.int32)
        docs[:40] = [3900, 4100]
        docs[155:160] = [700, 700]
        kw["doc_bounds"] = docs
    if "cap" in mods:
        kw.update(softcap=5.0, prefix_lens=np.array([3950, 0, 0, 100], np.int32),
                  alibi_slopes=(0.02 * 2.0 ** -np.arange(8)).astype(np.float32))
    check(x, **kw)


def test_more_rows_than_workspace_slots():
    """As many CTAs as fill the SMs: none is shared, and the workspace is not used."""
    x = build([130] * 40, [200 + i for i in range(40)], 8, 4, 64, "e4m3", 1800)
    check(x, max_seqlen_q=130)


def test_repeated_calls_are_bitwise_equal():
    x = build([1, 2, 30], [5000, 900, 300], 16, 2, 128, "e4m3", 1400)
    first = call(x)
    for _ in range(10):
        again = call(x)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h_q,h_kv,n", [(2, 2, 1), (12, 4, 1), (4, 4, 3), (4, 4, 33)])
def test_biased_calls_do_not_depend_on_the_calls_before(h_q, h_kv, n, d):
    """Row tiles with absent rows, behind calls that leave other slopes in shared memory."""
    x = build([n] * 3, [3000, 900, 400], h_q, h_kv, d, "int8", 1980 + d)
    slopes = np.exp2(-np.arange(h_q, dtype=np.float32))
    others = [(build([1] * 64, [2000] * 64, 8, 1, d, "int8", 1985), 1), (build([2] * 64, [2000] * 64, 8, 1, d, "int8", 1986), 2),
              (build([64] * 40, [200] * 40, 16, 4, d, "int8", 1987), LONG)]
    for hint in (1, LONG):
        seen = []
        for slope in (0.0, -1.0, -100.0, 0.0):
            for other, h in others:
                call(other, alibi_slopes=np.full(other["q"].shape[1], slope, np.float32), max_seqlen_q=h)
            seen.append(call(x, alibi_slopes=slopes, max_seqlen_q=hint))
        assert all(torch.equal(seen[0][0], s[0]) and torch.equal(seen[0][1], s[1]) for s in seen)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hint", [1, LONG])
def test_capped_scores_do_not_depend_on_what_stands_behind_the_length(hint, kind):
    """Scores of a few hundredths of the cap; the rows behind hold codes whose scores reach it."""
    x = build([1, 1, 3], [40, 100, 191], 8, 2, 128, kind, 1990, poison=False)
    clean = call(x, softcap=30.0, max_seqlen_q=hint)
    for r, n in enumerate(x["lens"]):
        b, row = x["table"][r, n // 64], n % 64
        for h in range(2):
            s = torch.sign(x["q"][x["cu"][r], 4 * h].float())
            x["kc"][b, h, row:] = (s * (448 if kind == "e4m3" else 127)).to(x["kc"].dtype)
    dirty = call(x, softcap=30.0, max_seqlen_q=hint)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


@pytest.mark.parametrize("hint", [1, LONG])
def test_a_captured_call_replays_on_new_inputs(hint):
    """A graph keeps its own scratch: replays beside eager calls, on another stream, give the eager results."""
    import sparse_mla_decoding_b200 as smla
    x = build([1, 2, 30], [3000, 900, 300], 16, 2, 128, "e4m3", 1500)
    t = {n: (x[n] if isinstance(x[n], torch.Tensor) else torch.from_numpy(x[n])).cuda()
         for n in ("q", "kc", "vc", "ks", "vs", "table", "lens", "cu")}

    def run():
        return smla.gqa_attention_with_kvcache(t["q"], t["kc"], t["vc"], t["ks"], t["vs"], t["table"], t["lens"],
                                               cu_seqlens_q=t["cu"], max_seqlen_q=hint)
    run()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        o, lse = run()
    q2 = t["q"].flip(0).contiguous()
    t["q"].copy_(q2)
    t["lens"].copy_(torch.tensor([1000, 890, 200], dtype=torch.int32))
    torch.cuda.synchronize()
    other = run()
    with torch.cuda.stream(side):
        graph.replay()
    beside = [run() for _ in range(3)]
    torch.cuda.synchronize()
    for a in [other] + beside:
        assert torch.equal(a[0], o) and torch.equal(a[1], lse)
    assert smla.paged_status()[0] == 0


@pytest.mark.parametrize("hint", [1, LONG])
def test_two_streams_at_once(hint):
    import sparse_mla_decoding_b200 as smla
    xs = [build([1, 1], [4000, 70], 8, 2, 128, kind, 1600) for kind in KINDS]
    ts = [{n: (x[n] if isinstance(x[n], torch.Tensor) else torch.from_numpy(x[n])).cuda()
           for n in ("q", "kc", "vc", "ks", "vs", "table", "lens", "cu")} for x in xs]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (t, s) in enumerate(zip(ts, streams)):
            with torch.cuda.stream(s):
                outs[i].append(smla.gqa_attention_with_kvcache(t["q"], t["kc"], t["vc"], t["ks"], t["vs"], t["table"],
                                                               t["lens"], cu_seqlens_q=t["cu"], max_seqlen_q=hint))
    torch.cuda.synchronize()
    for x, got in zip(xs, outs):
        U.compare(*got[0], reference(x))
        assert all(torch.equal(a[0], got[0][0]) and torch.equal(a[1], got[0][1]) for a in got)
