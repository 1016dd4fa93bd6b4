"""Compaction on the GPU, bit for bit, with every other token of the pool checked to be as it was."""
import numpy as np
import pytest
import torch

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
