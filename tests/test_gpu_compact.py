"""Compaction on the GPU, bit for bit, with every other token of the pool checked to be as it was."""
import numpy as np
import pytest
import torch

import _quant_ref as R
import _sparse_ref as S
import paged_kv_cache_302_gb300 as pa

pytestmark = pytest.mark.gpu


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def random_cache(g, NB, H, B, D, quant):
    """Random bits (nothing interprets them): (pool,) or (qpool, scales), on the host."""
    if quant:
        return (torch.randint(0, 256, (NB, H, 2, B, D), generator=g, dtype=torch.uint8),
                torch.randint(0, 256, (NB, H, 2, B), generator=g, dtype=torch.uint8))
    return (torch.randint(-2 ** 15, 2 ** 15, (NB, B, 2, H, D), generator=g, dtype=torch.int16).view(torch.float16),)


def token(c, blk, off):
    return tuple(x[blk, off] for x in c) if len(c) == 1 else tuple(x[blk, :, :, off] for x in c)


def move(c, tables, B, pairs):
    """Applies (source, destination) positions per sequence to host copies."""
    old = tuple(x.clone() for x in c)
    for s, src, dst in pairs:
        for x, y in zip(token(c, int(tables[s, dst // B]), dst % B), token(old, int(tables[s, src // B]), src % B)):
            x.copy_(y)


def run(c, tables, ctx, base, keeps, B, flag=0, moves=None):
    """Compacts device copies of c and compares all of them with the moves done on the host."""
    dev = [x.cuda() for x in c]
    bits = [x.view(torch.int16) if x.dtype == torch.float16 else x for x in c]
    err = err_word()
    ks = np.concatenate([[0], np.cumsum([len(k) for k in keeps])])
    pa.pa_compact_tokens(dev[0], tables.cuda(), i32(ctx), i32(base), i32(np.concatenate(keeps).astype(np.int32)), i32(ks),
                         dev_err=err, **({"scales": dev[1]} if len(c) == 2 else {}))
    if moves is None:
        moves = [(s, int(k), base[s] + j) for s, keep in enumerate(keeps) for j, k in enumerate(keep)]
    want = tuple(x.clone() for x in bits)
    move(want, tables, B, moves)
    for x, y in zip(dev, want):
        x = x.view(torch.int16) if x.dtype == torch.float16 else x
        assert torch.equal(x.cpu(), y)
    assert err.item() == flag


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("H, D, B", [(1, 64, 8), (2, 128, 16), (3, 64, 32), (8, 128, 16), (5, 128, 8), (40, 64, 16)])
def test_compaction(H, D, B, quant):
    """Random lists over a ragged batch: drafts' ends, halves of contexts, all kept, none kept, one kept."""
    g = torch.Generator().manual_seed(H + D + B)
    r = np.random.default_rng(H * D)
    ctx = [1, 7, 64, 500, 33, 1200, 90, 300]
    base = [0, 3, 64, 0, 32, 17, 60, 0]
    keeps = [[0], [6], [], np.sort(r.choice(500, 250, replace=False)), [], np.sort(r.choice(1183, 700, replace=False)) + 17,
             np.arange(60, 90), np.sort(r.choice(300, 299, replace=False))]
    MB = -(-max(ctx) // B) + 1
    NB = sum(-(-L // B) for L in ctx) + 4
    c = random_cache(g, NB, H, B, D, quant)
    run(c, S.make_tables(g, ctx, B, MB, NB), ctx, base, [np.asarray(k, dtype=np.int64) for k in keeps], B)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("gap", [1, 2, 63, 64, 65, 255, 256, 257, 1000])
def test_moves_by_a_constant_distance(gap, quant):
    """Every destination is a later token's source, at distances around the chunk's size."""
    g = torch.Generator().manual_seed(gap)
    L, B, H, D = 2500, 16, 2, 64
    c = random_cache(g, -(-L // B) + 2, H, B, D, quant)
    run(c, S.make_tables(g, [L], B, 160, c[0].shape[0]), [L], [0], [np.arange(gap, L)], B)


@pytest.mark.parametrize("quant", [False, True])
def test_bad_lists_are_flagged_and_not_followed(quant):
    g = torch.Generator().manual_seed(3)
    B, H, D, ctx = 8, 2, 64, [100, 100, 100]
    c = random_cache(g, 45, H, B, D, quant)
    tables = S.make_tables(g, ctx, B, 14, 45)
    good = np.arange(5, 100, 3)
    upto = lambda s, keep, n, b=0: [(s, int(k), b + j) for j, k in enumerate(keep[:n])]  # noqa: E731
    for keep, n in [(np.r_[np.arange(10, 40), 39, np.arange(41, 60)], 30),       # repeated
                    (np.r_[np.arange(10, 40), 20, np.arange(41, 60)], 30),       # descends
                    (np.r_[np.arange(10, 40), 100, 101], 30),                    # past the context
                    (np.r_[np.arange(10, 40), 2 ** 31 - 1], 30), (np.r_[-1, np.arange(10, 40)], 0),
                    (np.r_[np.arange(90, 100), -5, 99], 10)]:
        run(c, tables, ctx, [0, 0, 0], [good, keep, good], B, flag=pa.PA_DEV_ERR_CTX,
            moves=upto(0, good, 99) + upto(1, keep, n) + upto(2, good, 99))
    # a first position below base
    run(c, tables, ctx, [0, 6, 0], [good, good, good], B, flag=pa.PA_DEV_ERR_CTX, moves=upto(0, good, 99) + upto(2, good, 99))
    for base, lens in [([0, -1, 0], ctx), ([0, 0, 0], [100, -1, 100]), ([0, 0, 0], [100, 14 * B + 1, 100])]:
        run(c, tables, lens, base, [good, good, good], B, flag=pa.PA_DEV_ERR_CTX,
            moves=upto(0, good, 99) + upto(2, good, 99))


@pytest.mark.parametrize("quant", [False, True])
def test_tokens_without_a_block_stay_and_are_flagged(quant):
    g = torch.Generator().manual_seed(4)
    B, H, D, L = 8, 2, 64, 100
    c = random_cache(g, 20, H, B, D, quant)
    tables = S.make_tables(g, [L], B, 13, 20)
    keep = np.arange(5, 100, 3)
    t = tables.clone()
    t[0, 2], t[0, 7] = -1, 20
    moves = [(0, int(k), j) for j, k in enumerate(keep) if k // B not in (2, 7) and j // B not in (2, 7)]
    run(c, t, [L], [0], [keep], B, flag=pa.PA_DEV_ERR_BLOCK, moves=moves)


@pytest.mark.parametrize("quant", [False, True])
def test_entries_of_tokens_that_stay_are_not_looked_at(quant):
    g = torch.Generator().manual_seed(10)
    B, H, D, L = 8, 2, 64, 4000
    c = random_cache(g, 502, H, B, D, quant)
    tables = S.make_tables(g, [L], B, 500, 502)
    keep = np.r_[np.arange(16, 800), np.arange(900, 1000)]
    t = tables.clone()
    t[0, 2:90] = -1                                  # of tokens that are kept where they are
    run(c, t, [L], [16], [keep], B, moves=[(0, int(k), 800 + j) for j, k in enumerate(keep[784:])])
    t = tables.clone()
    t[0, 100:113] = -1                               # of the places that the others move to
    run(c, t, [L], [16], [keep], B, flag=pa.PA_DEV_ERR_BLOCK, moves=[])


def test_list_offsets_out_of_range_are_flagged():
    g = torch.Generator().manual_seed(5)
    B, H, D, ctx = 8, 1, 64, [50, 50, 50]
    c = random_cache(g, 24, H, B, D, False)
    tables = S.make_tables(g, ctx, B, 7, 24)
    keep = np.r_[np.arange(20, 30), np.arange(20, 30), np.arange(20, 30)]
    for ks, good in [([0, 10, 5, 15], [0]), ([0, 10, 20, 31], [0, 1]), ([-1, 10, 20, 30], [1, 2]),
                     ([0, 10, 2 ** 31 - 1, 2 ** 31 - 1], [0])]:
        pool = c[0].cuda()
        err = err_word()
        pa.pa_compact_tokens(pool, tables.cuda(), i32(ctx), i32([0, 0, 0]), i32(keep), i32(ks), dev_err=err)
        want = (c[0].view(torch.int16).clone(),)
        if ks == [0, 10, 5, 15]:                     # sequence 2's list is good: keep[5:15], whose order breaks at 10
            move(want, tables, B, [(0, 20 + j, j) for j in range(10)] + [(2, 25 + j, j) for j in range(5)])
        else:
            move(want, tables, B, [(s, 20 + j, j) for s in good for j in range(10)])
        assert torch.equal(pool.view(torch.int16).cpu(), want[0])
        assert err.item() == pa.PA_DEV_ERR_CTX


@pytest.mark.parametrize("quant", [False, True])
def test_blocks_past_32_bits_and_streams(quant):
    """A pool of more than 2^32 bytes, three sequences' lists, on a stream of its own and captured into a graph."""
    g = torch.Generator().manual_seed(6)
    B, H, D = 16, 8, 128
    NB = 140000 if quant else 70000
    ctx = [300, 77, 150]
    small = random_cache(g, 40, H, B, D, quant)
    big = [torch.empty((NB,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda") for x in small]
    at = torch.cat([torch.arange(20), torch.arange(NB - 20, NB)])
    for x, y in zip(big, small):
        x[at.cuda()] = y.cuda()
    low = S.make_tables(g, ctx, B, 19, 40)
    high = torch.where(low < 40, at[low.clamp(max=39).long()].to(torch.int32), low).cuda()
    r = np.random.default_rng(6)
    base = [0, 3, 100]
    keeps = [np.sort(r.choice(L - b, (L - b) // 2, replace=False)) + b for L, b in zip(ctx, base)]
    bits = tuple((x.view(torch.int16) if x.dtype == torch.float16 else x).clone() for x in small)
    moves = [(s, int(k), base[s] + j) for s, keep in enumerate(keeps) for j, k in enumerate(keep)]
    ks = np.cumsum([0] + [len(k) for k in keeps])
    args = (high, i32(ctx), i32(base), i32(np.concatenate(keeps)), i32(ks))
    kw = {"scales": big[1]} if quant else {}
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    pa.pa_compact_tokens(big[0], *args, stream=stream, **kw)
    with torch.cuda.graph(graph, stream=stream):
        pa.pa_compact_tokens(big[0], *args, **kw)
    graph.replay()
    torch.cuda.synchronize()
    for _ in range(2):
        move(bits, low, B, moves)
    for x, y in zip(big, bits):
        x = x[at.cuda()]
        assert torch.equal((x.view(torch.int16) if x.dtype == torch.float16 else x).cpu(), y)


@pytest.mark.parametrize("quant", [False, True])
def test_many_short_lists_and_one_long(quant):
    g = torch.Generator().manual_seed(7)
    B, H, D = 8, 2, 64
    ctx = [40] * 600 + [9000]
    r = np.random.default_rng(7)
    base = [int(r.integers(0, 30)) for _ in ctx[:-1]] + [10]
    keeps = [np.sort(r.choice(L - b, int(r.integers(0, min(12, L - b))), replace=False)) + b
             for L, b in zip(ctx[:-1], base)] + [np.sort(r.choice(8990, 6000, replace=False)) + 10]
    NB = sum(-(-L // B) for L in ctx) + 1
    run(random_cache(g, NB, H, B, D, quant), S.make_tables(g, ctx, B, 1130, NB), ctx, base, keeps, B)


@pytest.mark.parametrize("quant", [False, True])
def test_a_generation_with_drafts_forks_and_evictions(quant):
    """The calls as a server uses them: prompts written, summaries built, a fork, drafts appended and verified as a tree,
    the accepted ones compacted with the allocator's replacements, summaries of what changed rebuilt, a prefix evicted,
    blocks selected and attended -- against a plain list of every sequence's tokens."""
    H, G, D, B, top_k, MB = 2, 4, 64, 8, 6, 20
    gen = torch.Generator().manual_seed(8)
    r = np.random.default_rng(8)
    NB = 64
    alloc = pa.BlockAllocator(NB, B)
    pool = torch.zeros(NB, B, 2, H, D, dtype=torch.bfloat16, device="cuda")
    if quant:
        cache = (torch.zeros(NB, H, 2, B, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                 torch.zeros(NB, H, 2, B, dtype=torch.uint8, device="cuda"))
    else:
        cache = (pool,)
    kw = {"scales": cache[1]} if quant else {}
    box = torch.zeros(NB, H, 2, D, dtype=torch.int8, device="cuda")
    by = torch.zeros(NB, H, dtype=torch.uint8, device="cuda")
    tokens = {}                                          # sequence -> its K, V rows in order
    err = err_word()

    def copies(pairs):
        for x in cache + (box, by):
            if x.dtype == torch.int8 or x.dim() == 2:    # summaries are a block's like its tokens
                for a, b in np.asarray(pairs).tolist():
                    x[b] = x[a]
            elif len(pairs):
                pa.pa_copy_blocks(x, torch.from_numpy(np.ascontiguousarray(pairs)).cuda(), dev_err=err)

    def append(s, n):
        k, v = (torch.randn(n, H, D, generator=gen).bfloat16() for _ in range(2))
        slots, cow = alloc.append_slots(s, n)
        copies(cow)
        write = pa.pa_reshape_and_cache_quant if quant else pa.pa_reshape_and_cache
        write(k.cuda(), v.cuda(), *cache, torch.from_numpy(slots).cuda(), dev_err=err)
        tokens[s] = tokens.get(s, []) + [(k[i], v[i]) for i in range(n)]

    def tables(seqs):
        t, ctx = alloc.block_tables(seqs, MB)
        return torch.from_numpy(t).cuda(), torch.from_numpy(ctx).cuda()

    def summarize(seqs, n):
        t, ctx = tables(seqs)
        pa.pa_summarize_blocks(box, by, cache[0], t, ctx, max(max(n), 1), q_start=i32(np.cumsum([0] + list(n))),
                               dev_err=err, **kw)

    def compact(seqs, base, keeps):
        t, ctx = alloc.block_tables(seqs, MB)
        new = [b + len(k) for b, k in zip(base, keeps)]
        cow, upd = alloc.compact_batch(seqs, base, new, table_updates=True)
        copies(cow)
        t = torch.from_numpy(t).cuda()
        if len(upd):
            pa.pa_update_block_tables(t, torch.from_numpy(upd).cuda(), dev_err=err)
        pa.pa_compact_tokens(cache[0], t, torch.from_numpy(ctx).cuda(), i32(base), i32(np.concatenate(keeps)),
                             i32(np.cumsum([0] + [len(k) for k in keeps])), dev_err=err, **kw)
        for s, b, k in zip(seqs, base, keeps):
            tokens[s] = tokens[s][:b] + [tokens[s][i] for i in k]
        summarize(seqs, [n - b for n, b in zip(new, base)])

    def check(seqs):
        """Every sequence's tokens in the pool, its summaries, the selection by them, and the attention."""
        t, ctx = tables(seqs)
        q = torch.randn(len(seqs), H * G, D, generator=gen).bfloat16()
        sel = torch.empty(len(seqs), H, top_k, dtype=torch.int32, device="cuda")
        pa.pa_select_blocks(sel, q.cuda(), box, by, t, ctx, MB * B, B, dev_err=err)
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        pa.pa_decode_sparse(out, q.cuda(), cache[0], t, ctx, sel, dev_err=err, **kw)
        host, bb, ss = S.host_cache(cache), box.cpu().numpy(), by.cpu().numpy()
        for i, s in enumerate(seqs):
            L, blocks = len(tokens[s]), alloc.block_table(s)
            assert alloc.seq_len(s) == L == int(ctx[i])
            for h in range(H):
                k, v, ev = S.keys_of(host, blocks, h, L)
                want = np.stack([x[0][h].double().numpy() for x in tokens[s]])
                if quant:
                    want = R.values(*R.quantise(want))
                assert np.array_equal(k, want)
                x = np.array([S.box(k[b * B: b * B + B])[0] for b in range(len(blocks))])
                assert np.array_equal(bb[blocks, h], x)
                rows = slice(h * G, h * G + G)
                pick = S.select(S.scores(R.to64(q[i, rows]), bb[blocks, h], ss[blocks, h]), top_k, 1, 1)
                assert np.array_equal(sel[i, h].cpu().numpy(), pick)
                at = np.concatenate([np.arange(b * B, min(L, b * B + B)) for b in pick if b >= 0])
                want, tol = R.attend(R.to64(q[i, rows]), k[at], v[at], ev[at], np.ones((G, len(at)), bool), 1 / 8, True, quant)
                R.close(out[i, rows], want, tol, "attention")
        assert err.item() == 0

    for s, n in enumerate((50, 7, 90)):
        alloc.add_seq(s)
        append(s, n)
    summarize([0, 1, 2], [50, 7, 90])
    check([0, 1, 2])
    alloc.fork(0, 3)
    tokens[3] = list(tokens[0])
    check([0, 1, 2, 3])
    for _ in range(3):                                   # drafts, some of them accepted
        seqs = [0, 1, 2, 3]
        base = [len(tokens[s]) for s in seqs]
        for s in seqs:
            append(s, 9)
        keeps = [np.sort(r.choice(9, int(r.integers(0, 6)), replace=False)) + b for b in base]
        compact(seqs, base, keeps)
        check(seqs)
    alloc.fork(2, 4)
    tokens[4] = list(tokens[2])
    L = len(tokens[2])                                   # eviction from shared blocks: 4 keeps what it has
    compact([2, 0], [4, 10], [np.sort(r.choice(L - 4, L // 2, replace=False)) + 4, np.arange(10, 30)])
    check([0, 1, 2, 3, 4])
    for s in (0, 2, 4):
        append(s, 1)
    summarize([0, 2, 4], [1, 1, 1])
    check([0, 1, 2, 3, 4])
    for s in range(5):
        alloc.free_seq(s)
    assert alloc.num_free() == NB


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("base", [21, 24, 3])
def test_summaries_after_drafts_of_which_nothing_is_kept(base, quant):
    """Drafts written and summarised, none accepted (or a context cut back further): the header's procedure, a chunk of 1
    where base lies inside a block, makes every box its tokens' again.  A fork that is cut back leaves the box of the block it
    still shares as the longer sequence needs it."""
    H, D, B, NB, MB = 2, 64, 8, 24, 8
    gen = torch.Generator().manual_seed(base)
    alloc = pa.BlockAllocator(NB, B)
    if quant:
        cache = (torch.zeros(NB, H, 2, B, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                 torch.zeros(NB, H, 2, B, dtype=torch.uint8, device="cuda"))
    else:
        cache = (torch.zeros(NB, B, 2, H, D, dtype=torch.bfloat16, device="cuda"),)
    kw = {"scales": cache[1]} if quant else {}
    box = torch.zeros(NB, H, 2, D, dtype=torch.int8, device="cuda")
    by = torch.zeros(NB, H, dtype=torch.uint8, device="cuda")
    err = err_word()

    def append(s, n, size):
        slots, cow = alloc.append_slots(s, n)
        for x in cache if len(cow) else ():
            pa.pa_copy_blocks(x, torch.from_numpy(np.ascontiguousarray(cow)).cuda(), dev_err=err)
        k, v = ((size * torch.randn(n, H, D, generator=gen)).bfloat16().cuda() for _ in range(2))
        write = pa.pa_reshape_and_cache_quant if quant else pa.pa_reshape_and_cache
        write(k, v, *cache, torch.from_numpy(slots).cuda(), dev_err=err)

    def summarize(s, n):
        t, ctx = alloc.block_tables([s], MB)
        pa.pa_summarize_blocks(box, by, cache[0], torch.from_numpy(t).cuda(), torch.from_numpy(ctx).cuda(), max(n, 1),
                               q_start=i32([0, n]), dev_err=err, **kw)

    def as_defined(s):
        """Per block and head, whether its summary is that of the sequence's tokens."""
        blocks, L = alloc.block_table(s), alloc.seq_len(s)
        res = []
        for b, blk in enumerate(blocks):
            for h in range(H):
                want, e = S.box(S.keys_of(S.host_cache(cache), [blk], h, min(B, L - b * B))[0])
                res.append(np.array_equal(box[blk, h].cpu().numpy(), want) and by[blk, h].item() == e)
        return np.array(res)

    alloc.add_seq(0)
    append(0, 24 if base == 24 else 21, 1.0)
    summarize(0, alloc.seq_len(0))
    alloc.fork(0, 1)
    append(0, 9, 50.0)
    summarize(0, 9)
    assert as_defined(0).all()
    cow = alloc.compact_batch([0], [base], [base])
    assert len(cow) == 0 and alloc.seq_len(0) == base
    shared = base == 3                               # the first block is the fork's too
    if base % B and not shared:
        assert not as_defined(0).all()               # nothing kept, nothing rebuilt by a chunk of 0
        summarize(0, 1)
    if not shared:
        assert as_defined(0).all()
    assert as_defined(1).all()                       # (the shared block's box covers both sequences' tokens)
    alloc.fork(1, 2)
    alloc.compact_batch([2], [18], [18])
    assert as_defined(1).all() and err.item() == 0
