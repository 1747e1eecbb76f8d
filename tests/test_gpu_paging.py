"""Block tables, slot maps and the block-scaled cache's writer on the GPU, and a
serving step made of them: tables, writer, attention, for the block-scaled cache and
for the MLA cache."""
import numpy as np
import pytest
import torch

import paged_util as U

pytestmark = pytest.mark.gpu

BLOCK = U.BLOCK


# --------------------------------------------------------------------------- block tables
def tables(lens, new, free, num_free=None, max_new=None, cols=None):
    import sparse_mla_decoding_b200 as smla
    lens, new, free = (np.asarray(a, np.int32) for a in (lens, new, free))
    num_free = len(free) if num_free is None else num_free
    total = int(np.maximum(new, 0).sum())
    max_new = total if max_new is None else max_new
    cols = int((-(-(lens + np.maximum(new, 0)) // BLOCK)).max(initial=0)) + 1 if cols is None else cols
    rng = np.random.default_rng(3)
    table = rng.integers(0, 1 << 20, (len(lens), cols)).astype(np.int32)
    ref = U.extend_block_table(table, lens, new, free, num_free, max_new)
    t = torch.from_numpy(table).cuda()
    args = [torch.from_numpy(a).cuda() for a in (lens, new, free)]
    have = torch.tensor([num_free], dtype=torch.int32, device="cuda")
    for _ in range(2):                       # a call may be repeated
        slots, cu, out, left = smla.extend_block_table(t, *args, have, max_new)
    for got, want in zip((t, slots, cu, out), ref):
        assert got.dtype == torch.from_numpy(want).dtype and np.array_equal(got.cpu().numpy(), want)
    assert int(left) == ref[4]


@pytest.mark.parametrize("b", [1, 2, 31, 1000, 1024, 1025, 2500])
@pytest.mark.parametrize("most", [1, 300])
def test_tables_of_many_requests(b, most):
    rng = np.random.default_rng(b + most)
    lens = rng.integers(0, 400, b)
    new = np.full(b, 1) if most == 1 else rng.integers(0, most, b)
    need = (-(-(lens + new) // BLOCK) + (-lens // BLOCK)).sum()
    tables(lens, new, rng.permutation(int(need) + 9) + 5000)


def test_tables_around_block_edges():
    lens = np.repeat([0, 1, 63, 64, 65, 127, 128], 5)
    new = np.tile([0, 1, 63, 64, 130], 7)
    tables(lens, new, np.arange(1000)[::-1])


def test_one_long_prompt():
    tables([5], [150001], np.random.default_rng(0).permutation(3000))


def test_requests_that_do_not_fit():
    """The free list runs out, later requests that need nothing still get their rows; a full row, a full slot map."""
    tables([60, 60, 60, 10], [10, 10, 10, 3], [7, 8])
    tables([0, 0], [100, 30], [7, 8, 9], num_free=0)
    tables([0, 70, 10], [200, 5, 100], np.arange(50), cols=2)
    tables([0, 0, 0], [40, 40, 40], np.arange(50), max_new=100)
    tables([3, 4], [2, 2], np.arange(5), max_new=9)
    tables([10, 5], [-3, 4], np.arange(5))


def test_lengths_at_the_end_of_32_bits():
    """A row of 2^25 + 1 blocks: tokens up to position 2^31 - 2 get their rows, in the last block
    held or in a fresh one, and a length of 2^31 is declined."""
    import sparse_mla_decoding_b200 as smla
    top = 1 << 31
    cols = (1 << 25) + 1
    table = torch.full((1, cols), -1, dtype=torch.int32, device="cuda")
    table[0, (1 << 25) - 2:(1 << 25)] = torch.tensor([500, 600], dtype=torch.int32)
    table[0, (1 << 25) - 1:] = torch.tensor([600, -1], dtype=torch.int32)
    free = torch.tensor([7, 8], dtype=torch.int32, device="cuda")
    for length, new, fits in ((top - 63, 10, True), (top - 63, 62, True), (top - 70, 3, True), (top - 64, 63, True),
                              (top - 63, 63, False), (top - 5, 10, False), (top - 1, 70, False), (top - 1, 0, True)):
        t = table.clone()
        args = [torch.tensor([a], dtype=torch.int32, device="cuda") for a in (length, new, 2)]
        slots, cu, out, left = smla.extend_block_table(t, args[0], args[1], free, args[2], 70)
        held = -(-length // BLOCK)                    # the entries before this one are the request's
        need = -(-(length + new) // BLOCK) - held if fits else 0
        want = [-1] * 70
        if fits:
            pages = {(1 << 25) - 2: 500, (1 << 25) - 1: 600 if held == 1 << 25 else 8}
            want[:new] = [pages[p // BLOCK] * BLOCK + p % BLOCK for p in range(length, length + new)]
        assert slots.tolist() == want
        assert cu.tolist() == [0, new] and int(out) == length + (new if fits else 0) and int(left) == 2 - need
        ref = table[0, -3:].tolist()
        if need:
            ref[held - (cols - 3)] = 8
        assert t[0, -3:].tolist() == ref and torch.equal(t[0, :-3], table[0, :-3])


def test_shortened_requests_give_their_blocks_back():
    """Draft tokens are taken back across block edges and a request ends: the caller puts the
    entries behind the kept length on the free list, and after each step every block is held by
    one request or free."""
    import sparse_mla_decoding_b200 as smla
    rng = np.random.default_rng(12)
    nb, b, cols = 40, 4, 12
    table = torch.zeros(b, cols, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(nb).astype(np.int32)).cuda()
    left = torch.tensor([nb], dtype=torch.int32, device="cuda")
    lens = torch.zeros(b, dtype=torch.int32, device="cuda")
    col = torch.arange(cols, device="cuda")[None]
    for step in range(30):
        new = torch.from_numpy(rng.integers(0, 90, b).astype(np.int32)).cuda()
        _, _, lens, left = smla.extend_block_table(table, lens, new, free, left, 400)
        keep = lens - torch.from_numpy(rng.integers(0, 130, b).astype(np.int32)).cuda()
        keep = torch.where(torch.arange(b, device="cuda") == step % b, 0, keep.clamp(min=0)).to(torch.int32)
        gone = (col >= (keep[:, None] + 63) // 64) & (col < (lens[:, None] + 63) // 64)
        back = table[gone]
        free[int(left):int(left) + len(back)] = back
        left, lens = left + len(back), keep
        held = table[col < (lens[:, None] + 63) // 64]
        assert sorted(held.tolist() + free[:int(left)].tolist()) == list(range(nb))


def test_empty_batches():
    tables(np.zeros(0), np.zeros(0), np.arange(3), cols=1)
    tables(np.zeros(0), np.zeros(0), np.arange(3), cols=1, max_new=70)
    tables([3, 0], [0, 0], [])


# --------------------------------------------------------------------------- the writer
def pow2_scale(amax, kind):
    """The smallest power of two (>= 2^-126) at which amax fits the codes."""
    if amax == 0:
        return 0.0
    top = 448.0 if kind == "e4m3" else 127.0
    k = -126
    while amax / 2.0 ** k > top:
        k += 1
    return 2.0 ** k


def to_codes(x, kind):
    """x (float64; exact in float32 where it comes from a power-of-two scale) as codes."""
    if kind == "e4m3":
        return torch.from_numpy(x).clamp(-448, 448).to(torch.float32).to(torch.float8_e4m3fn)
    return torch.from_numpy(np.clip(np.rint(np.nan_to_num(x, nan=0.0, posinf=127, neginf=-127)), -127, 127)).to(torch.int8)


def write_reference(x, cu, old, table, codes, scale, kind):
    """codes [num_blocks, h, 64, d] and scale updated in place, one (block, head) at a time."""
    raw = codes.view(torch.int8)
    for r in range(len(old)):
        n = int(cu[r + 1] - cu[r])
        for b in range(int(old[r]) // BLOCK, -(-(int(old[r]) + n) // BLOCK) if n else 0):
            row0 = max(int(old[r]) - b * BLOCK, 0)
            t0 = b * BLOCK + row0 - int(old[r])
            rows = min(BLOCK - row0, n - t0)
            page = int(table[r, b])
            for h in range(x.shape[1]):
                new = x[cu[r] + t0:cu[r] + t0 + rows, h].double().numpy()
                was = float(scale[page, h]) if row0 else 0.0
                fine = np.abs(new[np.isfinite(new)])
                now = max(pow2_scale(fine.max(initial=0.0), kind), was)
                if was < now:
                    f = codes[page, h, :row0].double().numpy() * (was / now)
                    raw[page, h, :row0] = to_codes(f, kind).view(torch.int8)
                # float32 division, as the entry point defines the codes of a scale that is no power of two
                y = (new.astype(np.float32) / np.float32(now)).astype(np.float64) if now else np.zeros_like(new)
                raw[page, h, row0:row0 + rows] = to_codes(y, kind).view(torch.int8)
                scale[page, h] = now


def write_case(old, new, h, d, kind, seed, size=1.0):
    rng = np.random.default_rng(seed)
    old, new = np.asarray(old, np.int32), np.asarray(new, np.int32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    table, blocks = U.make_table(old + new, seed)
    sides = []
    for i in range(2):
        g = torch.Generator().manual_seed(seed + i)
        x = torch.randn(int(cu[-1]), h, d, generator=g) * torch.exp(torch.randn(int(cu[-1]), h, 1, generator=g))
        codes, _, _ = U.make_cache(blocks, h, d, kind, seed + 5 + i)
        scale = torch.from_numpy(2.0 ** rng.integers(-9, -3, (blocks, h))).float()
        sides.append([(x * size).to(torch.bfloat16), codes, scale])
    return old, new, cu, table, sides


def write(old, new, cu, table, sides, **kw):
    import sparse_mla_decoding_b200 as smla
    (k, kc, ks), (v, vc, vs) = [[t.cuda() for t in s] for s in sides]
    smla.quantize_kv_blocks(k, v, kc, vc, ks, vs, *(torch.from_numpy(a).cuda() for a in (table, old, old + new, cu)),
                            **kw)
    return [(kc.cpu(), ks.cpu()), (vc.cpu(), vs.cpu())]


def check_write(case, kind, **kw):
    old, new, cu, table, sides = case
    got = write(*case, check_device_status=True, **kw)
    for (codes, scale), (x, c, s) in zip(got, sides):
        c, s = c.clone(), s.clone()
        write_reference(x, cu, old, table, c, s, kind)
        assert torch.equal(scale, s)
        assert torch.equal(codes.view(torch.int8), c.view(torch.int8))   # untouched rows and blocks among them


KINDS = ["e4m3", "int8"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_writes_are_exact(d, kind):
    """First tokens, appends inside, up to and across blocks, several blocks, no tokens."""
    old = [0, 0, 0, 1, 63, 64, 65, 10, 40, 0, 127]
    new = [1, 64, 65, 1, 1, 1, 64, 5, 300, 0, 2]
    check_write(write_case(old, new, 3, d, kind, 10 + d), kind)


@pytest.mark.parametrize("kind", KINDS)
def test_many_requests(kind):
    rng = np.random.default_rng(5)
    check_write(write_case(rng.integers(0, 200, 300), rng.integers(0, 4, 300), 2, 64, kind, 20), kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1e-3, 1e3, 1e-39, 1e36])
def test_sizes(size, kind):
    """Growing and shrinking values beside older ones; the ends of bf16's range."""
    check_write(write_case([0, 30, 64], [70, 20, 3], 2, 64, kind, 30, size), kind)


@pytest.mark.parametrize("kind", KINDS)
def test_special_values(kind):
    case = write_case([0, 20], [64, 10], 2, 64, kind, 40)
    for x, codes, scale in case[4]:
        x[:, 0] = 0                                   # an all-zero head: scale 0 on a fresh block
        x[3, 1, 5], x[4, 1, 6], x[5, 1, 7] = float("inf"), float("-inf"), float("nan")
        x[66, 1] = float("inf")
        x[10, 1, 0] = 448.0
        scale[int(case[3][1, 0]), 1] = 0.3            # an older scale that is no power of two, and stays
    case[4][0][0][64:, 1] = 0.01
    check_write(case, kind)


def test_nan_tokens_in_a_block_of_zeros():
    """e4m3 has a code for them; int8 has none and stores 0."""
    for kind in KINDS:
        case = write_case([0, 20], [64, 10], 2, 64, kind, 45)
        old, new, cu, table, sides = case
        for x, codes, scale in sides:
            x[:, 0] = 0
            x[5, 0, 7] = x[6, 0, 8] = float("nan")
            x[8, 0, 1], x[9, 0, 2] = float("inf"), float("-inf")
        (kc, ks), (vc, vs) = write(*case, check_device_status=True)
        for codes, scale in ((kc, ks), (vc, vs)):
            page = int(table[0, 0])
            assert scale[page, 0] == 0
            got = codes[page, 0].float()
            nan = torch.zeros(64, 64, dtype=torch.bool)
            if kind == "e4m3":
                nan[5, 7] = nan[6, 8] = True
            assert torch.equal(torch.isnan(got), nan) and (got[~nan] == 0).all()


def test_ungranted_requests_are_left_alone():
    old, new, cu, table, sides = write_case([10, 20, 30], [3, 4, 5], 2, 64, "int8", 50)
    import sparse_mla_decoding_b200 as smla
    (k, kc, ks), (v, vc, vs) = [[t.cuda() for t in s] for s in sides]
    after = old + new
    after[1] = old[1]                                 # request 1 got no room
    smla.quantize_kv_blocks(k, v, kc, vc, ks, vs, *(torch.from_numpy(a).cuda() for a in (table, old, after, cu)),
                            check_device_status=True)
    for got, s, (x, c, sc) in ((kc, ks, sides[0]), (vc, vs, sides[1])):
        page = int(table[1, 0])
        assert torch.equal(got[page].cpu(), c[page]) and torch.equal(s[page].cpu(), sc[page])
        c, sc = c.clone(), sc.clone()
        keep = [0, 2]
        cu2 = [(cu[r], cu[r + 1]) for r in keep]
        x2 = torch.cat([x[a:b] for a, b in cu2])
        write_reference(x2, np.array([0, 3, 8]), old[keep], table[keep], c, sc, "int8")
        assert torch.equal(got.cpu(), c) and torch.equal(s.cpu(), sc)


def test_strided_tokens_and_blocks():
    import sparse_mla_decoding_b200 as smla
    case = write_case([5, 60], [70, 9], 2, 128, "int8", 60)
    old, new, cu, table, sides = case
    ref = write(*case)
    total, nb = int(cu[-1]), sides[0][1].shape[0]
    fused = torch.zeros(total, 8, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, 4:6], fused[:, 6:8] = sides[0][0].cuda(), sides[1][0].cuda()
    both = torch.stack([sides[0][1], sides[1][1]], 1).cuda()
    scales = torch.stack([sides[0][2], sides[1][2]], 1).cuda()
    smla.quantize_kv_blocks(fused[:, 4:6], fused[:, 6:8], both[:, 0], both[:, 1], scales[:, 0], scales[:, 1],
                            *(torch.from_numpy(a).cuda() for a in (table, old, old + new, cu)))
    for i in range(2):
        assert torch.equal(both[:, i].cpu(), ref[i][0]) and torch.equal(scales[:, i].cpu(), ref[i][1])


def test_bad_blocks_and_offsets_are_skipped_and_flagged():
    import sparse_mla_decoding_b200 as smla
    smla.reset_paged_status()
    old, new, cu, table, sides = write_case([0, 0], [70, 3], 2, 64, "int8", 70)
    table[0, 1] = sides[0][1].shape[0]
    got = write(old, new, cu, table, sides)
    assert smla.paged_status() == (1, 2)
    for (codes, scale), (x, c, s) in zip(got, sides):
        assert not torch.equal(codes[int(table[0, 0])], c[int(table[0, 0])])
    smla.reset_paged_status()
    cu[1] = -5
    write(old, new, cu, table, sides)
    assert smla.paged_status()[1] & 4
    with pytest.raises(smla.SmlaError):
        write(old, new, cu, table, sides, check_device_status=True)
    smla.reset_paged_status()
    assert smla.paged_status() == (0, 0)


# --------------------------------------------------------------------------- a serving run
@pytest.mark.parametrize("kind", KINDS)
def test_serving_steps(kind):
    """Prompts, then single tokens, then a run of draft tokens: tables, writer and attention
    over the growing cache.  The attention is checked against the cache as written (exact),
    and against the tokens that went in, whose codes are off by at most half a code step of
    a scale that is at most twice what the block's largest value needs."""
    import sparse_mla_decoding_b200 as smla
    b, h_q, h_kv, d = 5, 8, 2, 128
    nb, cols = 60, 12
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(9)
    kc = torch.zeros(nb, h_kv, BLOCK, d, dtype=torch.int8, device=dev).view(U.CACHE_TYPES[kind])
    vc = torch.zeros_like(kc.view(torch.int8)).view(U.CACHE_TYPES[kind])
    ks, vs = torch.zeros(nb, h_kv, device=dev), torch.zeros(nb, h_kv, device=dev)
    table = torch.zeros(b, cols, dtype=torch.int32, device=dev)
    free = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    left = torch.tensor([nb], dtype=torch.int32, device=dev)
    lens = torch.zeros(b, dtype=torch.int32, device=dev)
    seen_k, seen_v = [[] for _ in range(b)], [[] for _ in range(b)]
    steps = [[100, 64, 1, 130, 0], [1, 1, 1, 1, 40], [1, 1, 0, 1, 1], [4, 4, 4, 4, 4]] + [[1] * b] * 3
    for new in steps:
        n = sum(new)
        new_lens = torch.tensor(new, dtype=torch.int32, device=dev)
        slots, cu, after, left = smla.extend_block_table(table, lens, new_lens, free, left, n)
        qkv = (torch.randn(n, h_q + 2 * h_kv, d, generator=g, device=dev) * 1.3).to(torch.bfloat16)
        q, k, v = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:]
        smla.quantize_kv_blocks(k, v, kc, vc, ks, vs, table, lens, after, cu, check_device_status=True)
        lens = after
        o, lse = smla.gqa_attention_with_kvcache(q, kc, vc, ks, vs, table, lens, cu_seqlens_q=cu,
                                                 max_seqlen_q=max(new), softcap=30.0, check_device_status=True)
        at = 0
        for r in range(b):
            seen_k[r].append(k[at:at + new[r]].cpu())
            seen_v[r].append(v[at:at + new[r]].cpu())
            at += new[r]
        host = [x.cpu() for x in (kc, ks, vc, vs)]
        K = host[0].double().numpy() * host[1].double().numpy()[:, :, None, None]
        V = host[2].double().numpy() * host[3].double().numpy()[:, :, None, None]
        T, L = table.cpu().numpy(), lens.cpu().numpy()
        U.compare(o, lse, U.attention(q.double().cpu().numpy(), K, V, T, L, cu.cpu().numpy(), softcap=30.0,
                                      v_scale=host[3].double().numpy()))
    assert lens.tolist() == [sum(s[r] for s in steps) for r in range(b)]
    assert int(left) == nb - sum(-(-int(x) // BLOCK) for x in lens)
    for X, scale, seen in ((K, host[1], seen_k), (V, host[3], seen_v)):
        for r in range(b):
            x = torch.cat(seen[r]).double().numpy()
            n = len(x)
            pages = T[r, :-(-n // BLOCK)]
            got = X[pages].transpose(0, 2, 1, 3).reshape(-1, h_kv, d)[:n]
            s = np.repeat(scale.double().numpy()[pages], BLOCK, 0)[:n][:, :, None]
            # e4m3: half a step is 2^-4 of the value, or 2^-10 scales below 2^-6 scales; a code that was
            # rescaled stays on the finer grid or is rounded once more there.  int8: half a code, and
            # once more for each doubling of the scale while the block filled (1/2 + 1/4 + ... < 1 in
            # its final scale).
            half = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) + 2.0 ** -10 * s if kind == "e4m3" else s
            assert (np.abs(got - x) <= half).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("first", [5, 50])
def test_a_declined_request_leaves_the_step_to_the_others(first, kind):
    """Tables, writer and attention of a step in which one request gets no blocks: its cache and
    length stay, nothing is flagged, and the others' results are theirs.  What its own rows of o
    hold means nothing (their tokens are in no cache)."""
    import sparse_mla_decoding_b200 as smla
    h_q, h_kv, d, dev = 8, 2, 64, "cuda"
    g = torch.Generator(device=dev).manual_seed(11)
    kc = torch.zeros(9, h_kv, BLOCK, d, dtype=torch.int8, device=dev).view(U.CACHE_TYPES[kind])
    vc = torch.zeros_like(kc.view(torch.int8)).view(U.CACHE_TYPES[kind])
    ks, vs = torch.zeros(9, h_kv, device=dev), torch.zeros(9, h_kv, device=dev)
    table = torch.zeros(3, 8, dtype=torch.int32, device=dev)
    free = torch.randperm(9, generator=g, device=dev).to(torch.int32)
    left = torch.tensor([5], dtype=torch.int32, device=dev)
    lens = torch.zeros(3, dtype=torch.int32, device=dev)
    for new in ([10, 20, 30], [first, 300, 4]):       # a block each, then room in it, no room, room in it
        new_lens, n = torch.tensor(new, dtype=torch.int32, device=dev), sum(new)
        slots, cu, after, left = smla.extend_block_table(table, lens, new_lens, free, left, n)
        qkv = torch.randn(n, h_q + 2 * h_kv, d, generator=g, device=dev).to(torch.bfloat16)
        q, k, v = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:]
        before = [x.clone() for x in (kc, vc, ks, vs)]
        smla.quantize_kv_blocks(k, v, kc, vc, ks, vs, table, lens, after, cu, check_device_status=True)
        lens = after
        o, lse = smla.gqa_attention_with_kvcache(q, kc, vc, ks, vs, table, lens, cu_seqlens_q=cu,
                                                 max_seqlen_q=max(new), check_device_status=True)
    assert lens.tolist() == [10 + first, 20, 34] and int(left) == 2
    at, page = [0, first, first + 300, first + 304], int(table[1, 0])
    assert cu.tolist() == at and (slots[at[1]:at[2]] == -1).all() and (slots[:at[1]] >= 0).all()
    for x, was in zip((kc, vc, ks, vs), before):
        assert torch.equal(x[page].view(torch.int8), was[page].view(torch.int8))
    host = [x.cpu() for x in (kc, ks, vc, vs)]
    K, V = (host[i].double().numpy() * host[i + 1].double().numpy()[:, :, None, None] for i in (0, 2))
    for r in (0, 2):
        rows = slice(at[r], at[r + 1])
        U.compare(o[rows], lse[rows], U.attention(q[rows].double().cpu().numpy(), K, V, table[r:r + 1].cpu().numpy(),
                                                  lens[r:r + 1].cpu().numpy(), np.array([0, at[r + 1] - at[r]]),
                                                  v_scale=host[3].double().numpy()))


def test_slot_map_drives_the_mla_cache():
    """The same tables and slots for the MLA cache: quantize_kv by slots, then the dense decode."""
    import oracle
    import parity_util as PU
    import sparse_mla_decoding_b200 as smla
    rng = np.random.default_rng(4)
    b, h_q, nb, cols = 3, 16, 20, 6
    table = torch.zeros(b, cols, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(nb).astype(np.int32)).cuda()
    left = torch.tensor([nb], dtype=torch.int32, device="cuda")
    lens = torch.zeros(b, dtype=torch.int32, device="cuda")
    cache = torch.zeros(nb, BLOCK, 656, dtype=torch.uint8, device="cuda")
    for new in ([100, 64, 1], [1, 1, 1], [1, 1, 63]):
        n = sum(new)
        slots, cu, lens, left = smla.extend_block_table(table, lens, torch.tensor(new, dtype=torch.int32).cuda(), free,
                                                        left, n + 5)      # a padded slot map
        latent = torch.randn(n + 5, 512, device="cuda").to(torch.bfloat16)
        rope = torch.randn(n + 5, 64, device="cuda").to(torch.bfloat16)
        smla.quantize_kv(latent, rope, cache, slots)
    q = torch.randn(b, 1, h_q, 576, device="cuda").to(torch.bfloat16)
    sm, ns, tp = smla.get_mla_metadata_dense(lens, h_q)
    o, lse = smla.flash_mla_dense_with_kvcache(q, cache, table, lens, sm, ns, tp, check_device_status=True)
    bits = q.cpu().view(torch.int16).numpy().view(np.uint16)
    ref = oracle.dense_decode(bits, cache.cpu().numpy(), oracle.KV_FP8, table.cpu().numpy(),
                              lens.cpu().numpy().astype(np.int32), True)
    PU.compare(o.float().cpu().numpy(), lse.cpu().numpy(), ref, "slot map")
