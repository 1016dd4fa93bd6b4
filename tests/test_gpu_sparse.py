"""Block-sparse decode on the GPU: key summaries and block selection number for number, attention over listed blocks
element by element against a 64-bit form, with poisoned memory wherever a call has no business."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _quant_ref as R
import _sparse_ref as S
import paged_kv_cache_302_gb300 as pa

pytestmark = pytest.mark.gpu
DT = R.TORCH_DT


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def scales_of(c):
    return {"scales": c[1]} if len(c) == 2 else {}


# ------------------------------------------------------------------------------------------------ summaries

def poisoned_boxes(NB, H, D):
    return (torch.full((NB, H, 2, D), 55, dtype=torch.int8, device="cuda"),
            torch.full((NB, H), 0xEE, dtype=torch.uint8, device="cuda"))


def want_boxes(host, tables, ctx, n, B, want):
    """Rebuilds the touched summaries in want = (boxes, bytes), both numpy."""
    for s, L in enumerate(ctx):
        if n[s] <= 0:
            continue
        for b in range((L - n[s]) // B, -(-L // B)):
            blk = int(tables[s, b])
            for h in range(want[0].shape[1]):
                k, _, _ = S.keys_of(host, [blk], h, min(B, L - b * B))
                want[0][blk, h], want[1][blk, h] = S.box(k)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H, D, B, ctx, chunk", [
    (1, 64, 8, [1], [1]), (2, 128, 16, [16, 17, 15, 1], [1, 1, 1, 1]), (3, 64, 32, [33, 100, 5, 64], [2, 40, 0, 64]),
    (8, 128, 16, [200, 31, 7, 512, 90], [200, 16, 7, 3, 64]), (5, 128, 8, [70, 8], [9, 8]),
    (40, 64, 16, [37, 2], [20, 2])])
def test_summaries(H, D, B, ctx, chunk, dtype, quant):
    g = torch.Generator().manual_seed(H * 100 + D + B)
    MB = -(-max(ctx) // B) + 2
    NB = sum(-(-L // B) for L in ctx) + 3
    c = S.make_cache(g, NB, H, B, D, dtype, quant)
    tables = S.make_tables(g, ctx, B, MB, NB)
    # what lies behind a context's end is garbage
    nan = 0x7F if quant else math.nan
    for s, L in enumerate(ctx):
        if L % B:
            blk = int(tables[s, L // B])
            if quant:
                c[0].view(torch.uint8)[blk, :, :, L % B:] = nan
            else:
                c[0][blk, L % B:] = nan
    box, by = poisoned_boxes(NB, H, D)
    want = box.cpu().numpy().copy(), by.cpu().numpy().copy()
    want_boxes(S.host_cache(c), tables, ctx, chunk, B, want)
    err = err_word()
    qs = i32(np.concatenate([[0], np.cumsum(chunk)]))
    pa.pa_summarize_blocks(box, by, c[0], tables.cuda(), i32(ctx), max(chunk), q_start=qs, dev_err=err, **scales_of(c))
    assert np.array_equal(box.cpu().numpy(), want[0]) and np.array_equal(by.cpu().numpy(), want[1]) and err.item() == 0
    # whole contexts
    want_boxes(S.host_cache(c), tables, ctx, ctx, B, want)
    pa.pa_summarize_blocks(box, by, c[0], tables.cuda(), i32(ctx), max(ctx), dev_err=err, **scales_of(c))
    assert np.array_equal(box.cpu().numpy(), want[0]) and np.array_equal(by.cpu().numpy(), want[1]) and err.item() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_summaries_of_special_keys(dtype):
    """Zeros, the type's extremes, bounds of the exponent on both sides, infinities, NaN in some and in all tokens."""
    D, B, fi = 64, 8, torch.finfo(DT[dtype])
    values = [0.0, fi.tiny, -fi.tiny, fi.smallest_normal, fi.max, -fi.max, 127.0, 127.5, 126.5, 254.0, 255.0, -127.0,
              -128.0, 2.0 ** -20, math.inf, -math.inf, math.nan, 63.5, 64.0]
    x = torch.zeros(len(values) + 3, B, 2, 1, D)
    for i, v in enumerate(values):
        x[i, :, 0, 0] = torch.linspace(-1, 1, B * D).view(B, D) * (abs(v) if math.isfinite(v) else 1.0) * 0.3
        x[i, i % B, 0, 0, 7] = v
    n = len(values)
    x[n, :, 0, 0, 3] = math.nan                     # a channel of NaN alone
    x[n, :, 0, 0, 4] = 2.5
    x[n + 1, :, 0] = math.nan                       # a block of NaN alone
    x[n + 2, :, 0, 0, 5] = math.inf                 # nothing but infinities in a channel
    x = x.to(DT[dtype])
    NB = x.shape[0]
    tables = torch.arange(NB, dtype=torch.int32).view(1, NB)
    box, by = poisoned_boxes(NB, 1, D)
    pa.pa_summarize_blocks(box, by, x.cuda(), tables.cuda(), i32([NB * B]), NB * B)
    with np.errstate(invalid="ignore"):
        for b in range(NB):
            want, e = S.box(R.to64(x[b, :, 0, 0]))
            assert by[b, 0].item() == e, b
            assert np.array_equal(box[b, 0].cpu().numpy(), want), b


def test_summaries_of_every_quantised_pattern():
    """All e4m3 patterns under scales across their range, bytes that no write produces among them."""
    D, B, NB = 128, 16, 40
    g = torch.Generator().manual_seed(5)
    qp = torch.randint(0, 256, (NB, 2, 2, B, D), generator=g, dtype=torch.uint8)
    sc = torch.randint(0, 256, (NB, 2, 2, B), generator=g, dtype=torch.uint8)
    sc[::2] = torch.randint(120, 132, sc[::2].shape, generator=g, dtype=torch.uint8)
    qp[:4] &= 0x8F                                  # small and subnormal values
    tables = torch.randperm(NB, generator=g).to(torch.int32).view(1, NB)
    box, by = poisoned_boxes(NB, 2, D)
    pa.pa_summarize_blocks(box, by, qp.cuda().view(torch.float8_e4m3fn), tables.cuda(), i32([NB * B]), NB * B,
                           scales=sc.cuda())
    for b in range(NB):
        for h in range(2):
            want, e = S.box(S.keys_of((qp.numpy(), sc.numpy()), [b], h, B)[0])
            assert by[b, h].item() == e and np.array_equal(box[b, h].cpu().numpy(), want)


def test_summaries_flag_and_leave_out_bad_sequences():
    D, B, NB, MB = 64, 8, 12, 3
    g = torch.Generator().manual_seed(1)
    c = S.make_cache(g, NB, 2, B, D, "bf16", False)
    tables = torch.arange(NB, dtype=torch.int32).view(4, MB)
    for ctx, qs, top, entry, flag, good in [
            ([8, 25, 8, 8], [0, 1, 2, 3, 4], 1, None, pa.PA_DEV_ERR_CTX, [0, 2, 3]),      # a context past MB * B
            ([8, 3, 8, 8], [0, 1, 6, 7, 8], 5, None, pa.PA_DEV_ERR_CTX, [0, 2, 3]),       # a chunk past its context
            ([8, 8, 8, 8], [0, 1, 4, 5, 6], 2, None, pa.PA_DEV_ERR_CTX, [0, 2, 3]),       # longer than max_q_len
            ([8, 8, 8, 8], [0, 1, 0, 1, 2], 2, None, pa.PA_DEV_ERR_CTX, [0, 2, 3]),       # q_start descends
            ([8, -3, 8, 8], None, 8, None, pa.PA_DEV_ERR_CTX, [0, 2, 3]),
            ([8, 0, 8, 8], None, 8, None, 0, [0, 2, 3]),                                   # nothing there is no error
            ([8, 8, 8, 8], None, 8, NB, pa.PA_DEV_ERR_BLOCK, [0, 2, 3]),
            ([8, 8, 8, 8], None, 8, -1, pa.PA_DEV_ERR_BLOCK, [0, 2, 3])]:
        t = tables.clone()
        if entry is not None:
            t[1, 0] = entry
        box, by = poisoned_boxes(NB, 2, D)
        want = box.cpu().numpy().copy(), by.cpu().numpy().copy()
        want_boxes(S.host_cache(c), t[good], [8, 8, 8], [1, 1, 1], B, want)
        err = err_word()
        pa.pa_summarize_blocks(box, by, c[0], t.cuda(), i32(ctx), top, q_start=None if qs is None else i32(qs),
                               dev_err=err)
        assert err.item() == flag
        assert np.array_equal(box.cpu().numpy(), want[0]) and np.array_equal(by.cpu().numpy(), want[1])


def test_summaries_flag_chunks_past_32_bits():
    """Offsets whose difference is 1 only modulo 2^32 are no chunk of one token."""
    D, B, NB = 64, 8, 4
    c = S.make_cache(torch.Generator().manual_seed(2), NB, 2, B, D, "bf16", False)
    for qs in ([2 ** 31 - 1, -2 ** 31], [-2 ** 31, 2 ** 31 - 1]):
        box, by = poisoned_boxes(NB, 2, D)
        err = err_word()
        pa.pa_summarize_blocks(box, by, c[0], torch.arange(NB, dtype=torch.int32, device="cuda").view(1, NB), i32([20]), 4,
                               q_start=i32(qs), dev_err=err)
        assert err.item() == pa.PA_DEV_ERR_CTX and (box == 55).all() and (by == 0xEE).all()


# ------------------------------------------------------------------------------------------------ selection

def check_select(q, box, by, tables, ctx, B, top_k, sink, recent, H, flag=0, max_ctx=None, ctx_flag=()):
    N, Hq, D = q.shape
    G = Hq // H
    sel = torch.full((N, H, top_k), 77, dtype=torch.int32, device="cuda")
    err = err_word()
    pa.pa_select_blocks(sel, q.cuda(), box.cuda(), by.cuda(), tables.cuda(), i32(ctx), max_ctx or max(max(ctx), 1), B,
                        sink_blocks=sink, recent_blocks=recent, dev_err=err)
    got = sel.cpu().numpy()
    for s, L in enumerate(ctx):
        for h in range(H):
            want = np.full(top_k, -1)
            if s not in ctx_flag:
                at = tables[s, : -(-L // B)].numpy()
                bad = (at < 0) | (at >= box.shape[0])
                at = np.where(bad, 0, at)
                x = S.scores(R.to64(q[s, h * G: (h + 1) * G]), box[at, h].numpy(), by[at, h].numpy())
                want = S.select(np.where(bad, -np.inf, x), top_k, sink, recent)
            assert np.array_equal(got[s, h], want), (s, h)
    assert err.item() == flag
    return sel


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H, G, D, B, ctx, top_k, sink, recent", [
    (1, 1, 64, 8, [1], 1, 0, 0), (1, 1, 64, 8, [9], 1, 0, 1), (2, 4, 128, 16, [16, 17, 400, 1000], 8, 1, 1),
    (3, 3, 64, 32, [1, 2000, 5000, 64], 17, 2, 3), (8, 7, 128, 16, [5000, 4097], 64, 1, 1),
    (8, 8, 128, 8, [3000, 130, 8000], 33, 0, 0), (5, 2, 128, 16, [700, 1500], 40, 20, 20),
    (2, 5, 64, 8, [20000, 123], 500, 4, 16), (1, 6, 128, 32, [40000], 1000, 1, 1),
    (1, 2, 64, 8, [70000], 300, 1, 2), (1, 1, 64, 8, [140000, 3], 2000, 1, 1), (8, 1, 64, 16, [700, 90, 3000] * 3, 9, 1, 1),
    (16, 2, 128, 8, [2000, 64] * 9, 30, 1, 0), (16, 1, 64, 32, [900] * 20, 5, 0, 1),
    (16, 2, 128, 8, [700, 2048, 9] * 7, 40, 1, 1), (40, 1, 64, 16, [4000, 33] * 5, 17, 2, 0)])
def test_selection(H, G, D, B, ctx, top_k, sink, recent, dtype):
    g = torch.Generator().manual_seed(H * 31 + D + len(ctx))
    MB = -(-max(ctx) // B) + 1
    NB = sum(-(-L // B) for L in ctx) + 2
    box, by = S.make_boxes(g, NB, H, D)
    tables = S.make_tables(g, ctx, B, MB, NB)
    q = torch.randn(len(ctx), H * G, D, generator=g).to(DT[dtype])
    check_select(q, box, by, tables, ctx, B, top_k, sink, recent, H)


def test_selection_breaks_ties_by_the_lower_block():
    """Few distinct boxes, so that most scores are equal, at every place of the cut."""
    D, B, nb = 64, 8, 700
    g = torch.Generator().manual_seed(2)
    few, _ = S.make_boxes(g, 3, 2, D)
    box = few[torch.randint(0, 3, (nb,), generator=g)]
    by = torch.full((nb, 2), 124, dtype=torch.uint8)
    tables = torch.arange(nb, dtype=torch.int32).view(1, nb)
    q = torch.randn(1, 4, D, generator=g).half()
    for top_k in (1, 2, 31, 32, 33, 230, 256, 300, 511, 512, 513, 699, 700, 701):
        check_select(q, box, by, tables, [nb * B - 3], B, top_k, min(1, top_k), 0, 2)
    # all equal: boxes of zeros, and a query of zeros
    check_select(q, torch.zeros_like(box), by, tables, [nb * B], B, 100, 1, 1, 2)
    check_select(torch.zeros_like(q), box, by, tables, [nb * B], B, 100, 1, 1, 2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_selection_by_special_queries(dtype):
    """Extremes, subnormals, ties of the rounding, infinities, NaN, heads of very different size, bounds of the exponent,
    boxes at the integers' ends under scale bytes across the range and outside it."""
    D, B, nb, fi = 128, 8, 300, torch.finfo(DT[dtype])
    g = torch.Generator().manual_seed(3)
    box, _ = S.make_boxes(g, nb, 1, D)
    box[:40] = 127
    box[40:80] = -127
    box[80:100, :, 0] = -127
    box[80:100, :, 1] = 127
    by = torch.randint(60, 190, (nb, 1), generator=g, dtype=torch.uint8)
    by[::3] = 120
    tables = torch.randperm(nb, generator=g).to(torch.int32).view(1, nb)
    rows = []
    for v in (fi.max, -fi.max, fi.tiny, fi.smallest_normal, 511.0, 512.0, 510.0, 0.5, math.inf, -math.inf, math.nan):
        r = torch.randn(D, generator=g) * (abs(v) if math.isfinite(v) else 1.0) * 0.2
        r[9] = v
        rows.append(r)
    rows.append(torch.arange(D) % 64 * 8.0 - 252 + 0.5)         # halves: ties to even
    rows.append(torch.full((D,), math.nan))
    rows.append(torch.full((D,), 511.0))
    for i in range(0, len(rows) - 1, 2):
        check_select(torch.stack(rows[i: i + 2])[None].to(DT[dtype]), box, by, tables, [nb * B], B, 50, 1, 1, 1)


def test_selection_flags():
    D, B, nb, H = 64, 8, 64, 2
    g = torch.Generator().manual_seed(4)
    box, by = S.make_boxes(g, 3 * nb, H, D)
    tables = torch.arange(3 * nb, dtype=torch.int32).view(3, nb)
    q = torch.randn(3, 4, D, generator=g).half()
    tables[1, 5], tables[1, 20], tables[2, 7] = 3 * nb, -1, 1 << 30
    check_select(q, box, by, tables, [nb * B] * 3, B, 16, 1, 1, H, flag=pa.PA_DEV_ERR_BLOCK)
    # more bad entries than the list has room to leave out: the lowest of them are listed
    for n in (nb - 20, nb - 17, nb - 14, nb - 3):
        t = tables.clone()
        t[0, 2: 2 + n] = -1
        check_select(q, box, by, t, [nb * B] * 3, B, 18, 1, 1, H, flag=pa.PA_DEV_ERR_BLOCK)
    tables = torch.arange(3 * nb, dtype=torch.int32).view(3, nb)
    for bad in (0, -5, nb * B + 1):
        check_select(q, box, by, tables, [500, bad, 300], B, 16, 1, 1, H, flag=pa.PA_DEV_ERR_CTX, ctx_flag=(1,),
                     max_ctx=nb * B + 8)
    check_select(q, box, by, tables, [500, 401, 300], B, 16, 1, 1, H, flag=pa.PA_DEV_ERR_CTX, ctx_flag=(0, 1),
                 max_ctx=400)


@pytest.mark.parametrize("N", [3, 700])              # one kernel, a cluster per row; two kernels
@pytest.mark.parametrize("lens, MB", [([40, 8, 128], 16), ([40, 8, 4000], 500)])
def test_selection_flags_entries_of_contexts_that_it_lists_whole(lens, MB, N):
    """Contexts of no more than top_k blocks, alone and beside a longer one: every entry is looked at, the last one too, and
    none behind the context."""
    D, B, H, top_k = 64, 8, 2, 16
    g = torch.Generator().manual_seed(5)
    box, by = S.make_boxes(g, MB, H, D)
    ctx = (lens * N)[:N]
    tables = torch.full((N, MB), -1, dtype=torch.int32)
    for s, L in enumerate(ctx):
        tables[s, : -(-L // B)] = torch.randperm(MB, generator=g)[: -(-L // B)].to(torch.int32)
    q = torch.randn(N, 4, D, generator=g).half()
    check_select(q, box, by, tables, ctx, B, top_k, 1, 1, H, max_ctx=MB * B)
    for s, b, entry in ((0, 0, MB), (0, 4, -1), (1, 0, 1 << 30), (N - 2, 0, -2 ** 31)):
        t = tables.clone()
        t[s, b] = entry
        check_select(q, box, by, t, ctx, B, top_k, 1, 1, H, flag=pa.PA_DEV_ERR_BLOCK, max_ctx=MB * B)


# ------------------------------------------------------------------------------------------------ attention

def random_lists(g, ctx, H, B, top_k, fill=1.0):
    """Lists [N, H, top_k] in random order with padding strewn in."""
    sel = torch.full((len(ctx), H, top_k), -1, dtype=torch.int32)
    for s, L in enumerate(ctx):
        nb = -(-L // B)
        for h in range(H):
            n = min(nb, max(1, int(top_k * fill)))
            pick = torch.randperm(nb, generator=g)[:n].to(torch.int32)
            at = torch.randperm(top_k, generator=g)[:n]
            sel[s, h, at] = pick
    return sel


def want_sparse(q, host, tables, ctx, sel, B, scale, dtype, quant):
    """Output rows and their bounds, in 64 bits; duplicates count as often as they stand."""
    N, Hq, D = q.shape
    H = sel.shape[1]
    G = Hq // H
    out, tol = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    for s, L in enumerate(ctx):
        nb = -(-L // B)
        for h in range(H):
            t = []
            for e in sel[s, h].tolist():
                if 0 <= e < nb:
                    t += range(e * B, min(L, e * B + B))
            k, v, ev = S.keys_of(host, tables[s, :nb].numpy(), h, L)
            k, v, ev = k[t], v[t], ev[t]
            rows = slice(h * G, (h + 1) * G)
            see = np.ones((G, len(t)), dtype=bool)
            out[s, rows], tol[s, rows] = R.attend(R.to64(q[s, rows]), k, v, ev, see, scale, True,
                                                  quant or dtype == "f16")
    return out, tol


@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H, G, D, B, ctx, top_k", [
    (1, 1, 64, 8, [1], 1), (1, 8, 128, 16, [17, 300], 5), (2, 4, 128, 16, [1000, 16, 555], 64),
    (3, 3, 64, 32, [100, 700, 31, 1], 9), (8, 7, 128, 16, [2000, 130], 40), (5, 2, 64, 8, [400, 2500], 257),
    (2, 5, 128, 32, [3000, 90, 1700], 70), (8, 1, 128, 8, [129] * 20, 12),
    (8, 4, 128, 16, [1, 900, 333, 50] * 6, 48), (7, 3, 64, 32, [40, 2000, 700] * 9, 50), (1, 2, 64, 8, [300] * 90, 70),
    (8, 4, 128, 16, [700, 90] * 9, 30), (4, 2, 64, 32, [600, 31, 200] * 25, 7), (16, 1, 128, 8, [200, 60, 500] * 11, 33),
    (16, 1, 64, 16, [500, 33] * 20, 9), (2, 4, 128, 16, [9000, 300, 5000], 300), (3, 2, 64, 32, [12000, 40], 160),
    (1, 7, 128, 8, [6000], 700), (40, 2, 64, 16, [600, 900] * 4, 40)])
def test_attention(H, G, D, B, ctx, top_k, dtype, quant, out32):
    g = torch.Generator().manual_seed(H * 13 + D + top_k)
    MB = -(-max(ctx) // B) + 1
    NB = sum(-(-L // B) for L in ctx) + 3
    c = S.make_cache(g, NB, H, B, D, dtype, quant)
    tables = S.make_tables(g, ctx, B, MB, NB)
    host = S.host_cache(c)
    for s, L in enumerate(ctx):                      # garbage behind the context
        if L % B:
            blk = int(tables[s, L // B])
            if quant:
                c[0].view(torch.uint8)[blk, :, :, L % B:] = 0x7F
            else:
                c[0][blk, L % B:] = math.nan
    q = torch.randn(len(ctx), H * G, D, generator=g).to(DT[dtype])
    sel = random_lists(g, ctx, H, B, top_k, fill=0.8)
    if len(ctx) > 1:
        sel[-1, 0] = -1                              # a list without a block: zeros
    out = torch.full(q.shape, math.nan, dtype=torch.float32 if out32 else DT[dtype], device="cuda")
    err = err_word()
    pa.pa_decode_sparse(out, q.cuda(), c[0], tables.cuda(), i32(ctx), sel.cuda(), dev_err=err, **scales_of(c))
    want, tol = want_sparse(q, host, tables, ctx, sel, B, 1 / math.sqrt(D), dtype, quant)
    R.close(out, want, tol, "sparse decode")
    assert err.item() == 0


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("top_k", [8, 600])          # in clusters; in runs
def test_attention_flags_and_skips_bad_entries(quant, top_k):
    H, G, D, B = 2, 4, 64, 16
    ctx = [100, 200, 90]
    g = torch.Generator().manual_seed(8)
    c = S.make_cache(g, 40, H, B, D, "bf16", quant)
    tables = S.make_tables(g, ctx, B, 13, 40)
    q = torch.randn(3, H * G, D, generator=g).bfloat16()
    sel = random_lists(g, ctx, H, B, top_k, fill=0.5)
    host = S.host_cache(c)

    def run(t, lens, lists, flag):
        out = torch.full(q.shape, 9.0, dtype=torch.float32, device="cuda")
        err = err_word()
        pa.pa_decode_sparse(out, q.cuda(), c[0], t.cuda(), i32(lens), lists.cuda(), dev_err=err, **scales_of(c))
        assert err.item() == flag
        return out

    bad = sel.clone()
    bad[0, 1, 3], bad[1, 0, 0], bad[2, 1, 7], bad[2, 0, 2] = 7, 13, 1 << 30, 2 ** 31 - 1
    want, tol = want_sparse(q, host, tables, ctx, bad, B, 1 / 8, "bf16", quant)
    R.close(run(tables, ctx, bad, pa.PA_DEV_ERR_BLOCK), want, tol, "entries past the context")
    t = tables.clone()
    t[1, 3], t[1, 5] = -1, 40                        # these blocks of sequence 1 cannot be read
    lists = sel.clone()
    lists[1, :, :4] = torch.tensor([3, 2, 5, 6], dtype=torch.int32)
    without = lists.clone()
    without[(without == 3) | (without == 5)] = torch.where(
        torch.arange(3).view(3, 1, 1) == 1, -1, lists)[(without == 3) | (without == 5)]
    want, tol = want_sparse(q, host, tables, ctx, without, B, 1 / 8, "bf16", quant)
    R.close(run(t, ctx, lists, pa.PA_DEV_ERR_BLOCK), want, tol, "entries without a block")
    want, tol = want_sparse(q, host, tables, ctx, sel, B, 1 / 8, "bf16", quant)
    for L in (0, -1, 13 * B + 1):
        out = run(tables, [100, L, 90], sel, pa.PA_DEV_ERR_CTX)
        assert (out[1] == 9.0).all()
        R.close(out[[0, 2]], want[[0, 2]], tol[[0, 2]], "the other sequences")


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("times", [1, 101])          # in clusters; in runs
def test_attention_counts_repeated_blocks_and_takes_lists_in_any_order(quant, times):
    H, G, D, B, ctx = 1, 4, 128, 16, [77]
    g = torch.Generator().manual_seed(9)
    c = S.make_cache(g, 8, H, B, D, "f16", quant)
    tables = S.make_tables(g, ctx, B, 5, 8)
    q = torch.randn(1, G, D, generator=g).half()
    sel = torch.tensor([4, 2, 4, -1, 0, 2, 2, -7] * times, dtype=torch.int32).view(1, 1, -1)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    pa.pa_decode_sparse(out, q.cuda(), c[0], tables.cuda(), i32(ctx), sel.cuda(), **scales_of(c))
    want, tol = want_sparse(q, S.host_cache(c), tables, ctx, sel, B, 1 / math.sqrt(D), "f16", quant)
    R.close(out, want, tol, "sparse decode")


@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N, L, top_k", [
    (3, 500, 20), (3, 9000, 600), (700, 60, 4)])     # in clusters; in runs, rows divided; in runs, most rows whole
def test_attention_with_nan_in_queries_and_keys(N, L, top_k, D, quant, out32):
    """A NaN in one head's query, in every listed key of a KV head, in one listed key: these rows are NaN and no other is;
    lists without a block give zeros beside them, NaN query or not."""
    H, G, B, NB = 2, 4, 16, 600
    g = torch.Generator().manual_seed(N + D)
    c = S.make_cache(g, NB, H, B, D, "bf16", quant)
    tables = torch.stack([torch.randperm(NB - 2, generator=g)[: -(-L // B)] for _ in range(N)]).to(torch.int32)
    q = torch.randn(N, H * G, D, generator=g).bfloat16()
    ctx = [L] * N
    sel = random_lists(g, ctx, H, B, top_k)
    sel[1, 1] = -1                                   # no block
    bad = torch.zeros(N, H * G, dtype=torch.bool)
    for s, h in ((0, 1), (1, 2), (1, 6), (N - 1, 0)):
        q[s, h, 5] = math.nan
        bad[s, h] = h != 6                           # (sequence 1's second KV head has no block)
    tables[2, :] = NB - 1                            # a sequence whose second KV head's keys are all NaN
    pick = sel[0, 1][sel[0, 1] >= 0][0].item()       # and one whose second KV head has one such key
    tables[0, pick] = NB - 2
    if quant:
        c[0].view(torch.uint8)[NB - 1, 1, 0, :, 3] = 0x7F
        c[0].view(torch.uint8)[NB - 2, 1, 0, 1, 9] = 0xFF
    else:
        c[0][NB - 1, :, 0, 1, 3] = math.nan
        c[0][NB - 2, 1, 0, 1, 9] = math.nan
    bad[2, G:] = bad[0, G:] = True
    out = torch.full(q.shape, 9.0, dtype=torch.float32 if out32 else q.dtype, device="cuda")
    err = err_word()
    pa.pa_decode_sparse(out, q.cuda(), c[0], tables.cuda(), i32(ctx), sel.cuda(), dev_err=err, **scales_of(c))
    assert err.item() == 0
    nan = out.isnan().cpu()
    assert torch.equal(nan.all(-1), bad) and torch.equal(nan.any(-1), bad)
    assert (out[1, G:] == 0).all()
    some = [0, 1, 2, N - 1]                          # the rows beside them
    for h in range(H):
        k = [S.keys_of(S.host_cache(c), tables[s].numpy(), h, L) for s in some]
        for i, s in enumerate(some):
            rows = [r for r in range(h * G, h * G + G) if not bad[s, r]]
            t = [x for e in sel[s, h].tolist() if e >= 0 for x in range(e * B, min(L, e * B + B))]
            if rows and t:
                want, tol = R.attend(R.to64(q[s, rows]), k[i][0][t], k[i][1][t], k[i][2][t], np.ones((len(rows), len(t)), bool),
                                     1 / math.sqrt(D), True, quant)
                R.close(out[s, rows], want, tol, "rows beside NaN")


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("H, D, B, ctx", [
    (1, 64, 8, [1]), (1, 128, 8, [33]), (2, 64, 16, [64]), (1, 64, 8, [97]), (1, 128, 16, [128]), (1, 64, 32, [129]),
    (1, 128, 8, [160]), (3, 64, 16, [96]), (2, 128, 32, [150, 1]), (3, 64, 8, [32, 96, 64, 31]), (1, 64, 16, [2300]),
    (1, 128, 8, [2100, 1, 2000])])
def test_attention_of_few_units_by_runs(H, D, B, ctx, quant):
    """Long lists over short contexts: fewer units than a run takes, one more, rows cut at every place."""
    G, top_k = 4, 300
    g = torch.Generator().manual_seed(sum(ctx) + D + B)
    MB, NB = -(-max(ctx) // B), sum(-(-L // B) for L in ctx) + 2
    c = S.make_cache(g, NB, H, B, D, "bf16", quant)
    tables = S.make_tables(g, ctx, B, MB, NB)
    q = torch.randn(len(ctx), H * G, D, generator=g).bfloat16()
    sel = torch.full((len(ctx), H, top_k), -1, dtype=torch.int32)
    for s, L in enumerate(ctx):
        for h in range(H):
            pick = torch.randperm(-(-L // B), generator=g)[:top_k].to(torch.int32)
            sel[s, h, : len(pick)] = pick
    out = torch.full(q.shape, math.nan, dtype=torch.float32, device="cuda")
    err = err_word()
    pa.pa_decode_sparse(out, q.cuda(), c[0], tables.cuda(), i32(ctx), sel.cuda(), dev_err=err, **scales_of(c))
    want, tol = want_sparse(q, S.host_cache(c), tables, ctx, sel, B, 1 / math.sqrt(D), "bf16", quant)
    R.close(out, want, tol, "sparse decode")
    assert err.item() == 0


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_every_block_listed_is_the_whole_decode(D, quant):
    H, G, B, ctx = 4, 4, 16, [1000, 33, 512]
    g = torch.Generator().manual_seed(10)
    NB = sum(-(-L // B) for L in ctx) + 1
    c = S.make_cache(g, NB, H, B, D, "bf16", quant)
    tables = S.make_tables(g, ctx, B, 63, NB).cuda()
    q = torch.randn(3, H * G, D, generator=g).bfloat16().cuda()
    box, by = poisoned_boxes(NB, H, D)
    pa.pa_summarize_blocks(box, by, c[0], tables, i32(ctx), max(ctx), **scales_of(c))
    sel = torch.empty(3, H, 70, dtype=torch.int32, device="cuda")
    pa.pa_select_blocks(sel, q, box, by, tables, i32(ctx), max(ctx), B)
    a, b = (torch.empty(q.shape, dtype=torch.float32, device="cuda") for _ in range(2))
    pa.pa_decode_sparse(a, q, c[0], tables, i32(ctx), sel, **scales_of(c))
    if quant:
        pa.pa_decode_quant(b, q, c[0], c[1], tables, i32(ctx), max(ctx))
    else:
        pa.pa_decode(b, q, c[0], tables, i32(ctx), max(ctx))
    # both are within the 64-bit form's bound; their difference is within twice that
    lists = [list(range(-(-L // B))) for L in ctx]
    ref = torch.full((3, H, 63), -1, dtype=torch.int32)
    for s, x in enumerate(lists):
        ref[s, :, : len(x)] = torch.tensor(x, dtype=torch.int32)
    want, tol = want_sparse(q.cpu(), S.host_cache(c), tables.cpu(), ctx, ref, B, 1 / math.sqrt(D), "bf16", quant)
    R.close(a, want, tol, "sparse decode")
    R.close(b, want, tol, "whole decode")


# ------------------------------------------------------------------------------------------------ the calls in use

class Step:
    """A batch with its cache, summaries and queries, and one decode step over it: rebuild, select, attend."""

    def __init__(self, seed, ctx, H, G, D, B, dtype, quant, top_k, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.H, self.B, self.D, self.top_k = ctx, H, B, D, top_k
        self.NB = sum(-(-L // B) for L in ctx) + 3
        self.cache = S.make_cache(g, self.NB, H, B, D, dtype, quant)
        self.tables = S.make_tables(g, ctx, B, -(-max(ctx) // B) + extra, self.NB).cuda()
        self.q = torch.randn(len(ctx), H * G, D, generator=g).to(DT[dtype]).cuda()
        self.dctx = i32(ctx)

    def buffers(self):
        N = len(self.ctx)
        nan = torch.full(self.q.shape, math.nan, dtype=self.q.dtype, device="cuda")
        return poisoned_boxes(self.NB, self.H, self.D) + (
            torch.full((N, self.H, self.top_k), -9, dtype=torch.int32, device="cuda"), nan,
            torch.full((pa.pa_select_workspace_bytes(N, self.H, max(self.ctx), self.B),), 0xFF, dtype=torch.uint8,
                       device="cuda"),
            torch.full((pa.pa_decode_sparse_workspace_bytes(N, self.q.shape[1], self.H, self.D, self.B, self.top_k),), 0xFF,
                       dtype=torch.uint8, device="cuda"))

    def run(self, b, stream=None):
        box, by, sel, out, ws1, ws2 = b
        kw = dict(stream=stream, **scales_of(self.cache))
        pa.pa_summarize_blocks(box, by, self.cache[0], self.tables, self.dctx, max(self.ctx), **kw)
        pa.pa_select_blocks(sel, self.q, box, by, self.tables, self.dctx, max(self.ctx), self.B, workspace=ws1,
                            stream=stream)
        pa.pa_decode_sparse(out, self.q, self.cache[0], self.tables, self.dctx, sel, workspace=ws2, **kw)
        return sel, out


SHAPES = [([3000, 700, 41, 1900] * 3, 2, 4, 64, 16, "f16", False, 20), ([5000] * 12, 8, 2, 128, 16, "bf16", True, 64),
          ([900, 20000], 4, 8, 128, 8, "bf16", False, 100), ([9000, 700, 41, 6000], 2, 4, 128, 16, "bf16", False, 300),
          ([9000, 700, 41, 6000] * 8, 4, 2, 64, 32, "f16", True, 150)]


@pytest.mark.parametrize("shape", SHAPES)
def test_steps_side_by_side_give_the_bits_they_give_alone(shape):
    """Three streams, each with buffers and workspaces of its own, poisoned before; and again with the library's own
    workspaces."""
    st = Step(3, *shape[:7], shape[7])
    sel, out = st.run(st.buffers())
    bufs = [st.buffers() for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in bufs]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, b in zip(streams, bufs):
            st.run(b, s)
    torch.cuda.synchronize()
    for b in bufs:
        assert torch.equal(b[2], sel) and torch.equal(b[3], out)
    bufs = [st.buffers()[:4] + (None, None) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, b in zip(streams, bufs):
            st.run(b, s)
    torch.cuda.synchronize()
    for b in bufs:
        assert torch.equal(b[2], sel) and torch.equal(b[3], out)


@pytest.mark.parametrize("shape", SHAPES)
def test_captured_step_follows_what_its_inputs_hold(shape):
    """One graph, replayed with other queries, lengths and tables in the same tensors."""
    st = Step(4, *shape[:7], shape[7])
    b = st.buffers()
    stream = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        st.run(b)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=stream):
            st.run(b)
    for seed in (0, 1, 2):
        r = np.random.default_rng(seed)
        st.q.copy_(torch.randn(st.q.shape, generator=torch.Generator().manual_seed(seed)))
        st.dctx.copy_(i32([int(r.integers(1, L + 1)) for L in st.ctx]))
        b[3].fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        sel, out = b[2].clone(), b[3].clone()
        fresh = st.buffers()
        fresh[0].copy_(b[0])
        fresh[1].copy_(b[1])
        st.run(fresh)
        assert torch.equal(sel, fresh[2]) and torch.equal(out, fresh[3])


@pytest.mark.parametrize("quant", [False, True])
def test_attention_over_a_list_of_nearly_2_31_tokens(quant):
    """As many tokens as block tables can name, through a table whose entries are all one block: the softmax over its tokens,
    the last five counting once less.  Each of a CTA's fp32 additions, four to a unit, is off by at most 2^-22 of the sum so
    far."""
    H, G, D, B, NB = 1, 2, 64, 16, 2
    MB = 2 ** 27 - 1
    L = MB * B - 5
    g = torch.Generator().manual_seed(17)
    c = S.make_cache(g, NB, H, B, D, "bf16", quant)
    q = torch.randn(1, G, D, generator=g).bfloat16()
    tables = torch.ones(1, MB, dtype=torch.int32, device="cuda")
    sel = torch.arange(MB, dtype=torch.int32, device="cuda").view(1, 1, MB)
    out = torch.full(q.shape, 1e9, device="cuda")
    err = err_word()
    pa.pa_decode_sparse(out, q.cuda(), c[0], tables, i32([L]), sel, dev_err=err, **scales_of(c))
    assert err.item() == 0
    k, v, ev = S.keys_of(S.host_cache(c), [1], 0, B)
    n = np.where(np.arange(B) < B - 5, MB, MB - 1.0)
    s = R.to64(q[0]) @ k.T / 8
    w = n * np.exp(s - s.max(axis=1, keepdims=True))
    want, mag = (w @ v) / w.sum(axis=1, keepdims=True), (w @ np.abs(v)) / w.sum(axis=1, keepdims=True)
    _, tol = R.attend(R.to64(q[0]), k, v, ev, np.ones((G, len(n)), bool), 1 / 8, True, quant)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    steps = 4 * 2 * (MB * B // 32 // (sms * 4) + 1)      # (four CTAs per SM or more; numerator and denominator)
    R.close(out[0], want, tol * 2 + steps * 2.0 ** -22 * mag, "long list")


def test_attention_into_pinned_host_memory():
    for ctx, quant in (([700, 90], False), ([500] * 40, True)):
        st = Step(5, ctx, 2, 4, 128, 16, "bf16", quant, 20)
        sel, out = st.run(st.buffers())
        host = torch.full(out.shape, math.nan, dtype=out.dtype).pin_memory()
        pa.pa_decode_sparse(host, st.q, st.cache[0], st.tables, st.dctx, sel, **scales_of(st.cache))
        torch.cuda.synchronize()
        assert torch.equal(host, out.cpu())


def test_workspaces_and_lists_at_odd_addresses():
    """Workspaces of the least size at odd multiples of 16 bytes inside a poisoned buffer, lists at odd multiples of four,
    scale bytes at odd ones: the same bits, and nothing beside them written."""
    for ctx in ([900, 3000, 15], [2000] * 30):
        st = Step(6, ctx, 2, 4, 64, 16, "bf16", False, 33)
        box, by, sel, out, ws1, ws2 = st.buffers()
        want = [x.clone() for x in st.run((box, by, sel, out, ws1, ws2))]
        n1, n2 = ws1.numel(), ws2.numel()
        base = torch.full((n1 + n2 + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        big_sel = torch.full((sel.numel() + 7,), -9, dtype=torch.int32, device="cuda")
        big_by = torch.full((by.numel() + 9,), 0xA5, dtype=torch.uint8, device="cuda")
        sel2, by2 = big_sel[3: 3 + sel.numel()].view(sel.shape), big_by[5: 5 + by.numel()].view(by.shape)
        b1, b2 = base[16: 16 + n1], base[n1 + 2048 - n1 % 16 + 16: n1 + 2048 - n1 % 16 + 16 + n2]
        box.fill_(0)
        got = st.run((box, by2, sel2, torch.full_like(out, math.nan), b1, b2))
        used = st.tables[st.tables < st.NB].long()       # (the others keep each buffer's own poison)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(by2[used], by[used])
        assert (big_sel[:3] == -9).all() and (big_sel[3 + sel.numel():] == -9).all()
        assert (big_by[:5] == 0xA5).all() and (big_by[5 + by.numel():] == 0xA5).all()
        assert (base[:16] == 0xA5).all() and (base[16 + n1: n1 + 2048 - n1 % 16 + 16] == 0xA5).all()
        assert (base[n1 + 2048 - n1 % 16 + 16 + n2:] == 0xA5).all()


@pytest.mark.parametrize("quant", [False, True])
def test_offsets_past_32_bits(quant):
    """Blocks at the far end of a pool of more than 2^32 bytes and (16 bit) 2^31 elements."""
    H, G, D, B, top_k = 8, 4, 128, 16, 6
    NB = 140000 if quant else 70000
    ctx = [150, 97]
    g = torch.Generator().manual_seed(11)
    small = S.make_cache(g, 24, H, B, D, "bf16", quant)
    big = tuple(torch.empty((NB,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda") for x in small)
    at = torch.cat([torch.arange(8), torch.arange(NB - 16, NB)])
    raw = lambda x: x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x  # noqa: E731
    for x, y in zip(big, small):
        raw(x)[at.cuda()] = raw(y)
    low = S.make_tables(g, ctx, B, 10, 24)
    high = torch.where(low < 24, at[low.clamp(max=23).long()].to(torch.int32), low)
    q = torch.randn(2, H * G, D, generator=g).bfloat16().cuda()
    res = []
    for cache, tables, nb in ((small, low.cuda(), 24), (big, high.cuda(), NB)):
        box = torch.zeros((nb, H, 2, D), dtype=torch.int8, device="cuda")
        by = torch.zeros((nb, H), dtype=torch.uint8, device="cuda")
        err = err_word()
        pa.pa_summarize_blocks(box, by, cache[0], tables, i32(ctx), 150, dev_err=err, **scales_of(cache))
        sel = torch.empty(2, H, top_k, dtype=torch.int32, device="cuda")
        pa.pa_select_blocks(sel, q, box, by, tables, i32(ctx), 150, B, dev_err=err)
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        pa.pa_decode_sparse(out, q, cache[0], tables, i32(ctx), sel, dev_err=err, **scales_of(cache))
        assert err.item() == 0
        res.append((sel, out))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_many_sequences():
    """More sequences than one pass over the lengths takes, bad ones among them, more rows than the device's CTAs."""
    N, H, G, D, B, top_k = 1500, 2, 2, 64, 8, 4
    r = np.random.default_rng(12)
    ctx = r.integers(1, 90, size=N)
    bad = r.choice(N, 40, replace=False)
    g = torch.Generator().manual_seed(12)
    NB = int(sum(-(-ctx // B))) + 1
    c = S.make_cache(g, NB, H, B, D, "f16", False)
    tables = S.make_tables(g, ctx.tolist(), B, 12, NB)
    lens = ctx.copy()
    lens[bad] = r.choice([0, -1, 97], size=40)
    q = torch.randn(N, H * G, D, generator=g).half()
    box, by = poisoned_boxes(NB, H, D)
    err = err_word()
    pa.pa_summarize_blocks(box, by, c[0], tables.cuda(), i32(ctx), 90, dev_err=err)
    assert err.item() == 0
    sel = check_select(q, box.cpu(), by.cpu(), tables, lens.clip(0, 97).tolist(), B, top_k, 1, 1, H,
                       flag=pa.PA_DEV_ERR_CTX, max_ctx=96, ctx_flag=set(bad.tolist()))
    out = torch.full(q.shape, 5.0, dtype=torch.float32, device="cuda")
    pa.pa_decode_sparse(out, q.cuda(), c[0], tables.cuda(), i32(lens), sel, dev_err=err)
    assert err.item() == pa.PA_DEV_ERR_CTX and (out[torch.from_numpy(bad)] == 5.0).all()
    good = np.setdiff1d(np.arange(N), bad)
    want, tol = want_sparse(q[good], S.host_cache(c), tables[good], ctx[good].tolist(), sel.cpu()[good], B, 1 / 8, "f16",
                            False)
    R.close(out[torch.from_numpy(good)], want, tol, "many sequences")


@pytest.mark.parametrize("rows", ["few", "many"])
def test_quantised_attention_with_queries_and_scales_of_extreme_size(rows):
    """bf16 queries from fp32's subnormal numbers to its largest, scale bytes at both ends: finite, and within bounds where
    the scores themselves fit fp32."""
    H, G, D, B, top_k = 1, 6, 128, 16, 8
    ctx = [130, 100] if rows == "few" else [130, 100] * 40
    g = torch.Generator().manual_seed(13)
    NB = sum(-(-L // B) for L in ctx) + 1
    c = S.make_cache(g, NB, H, B, D, "bf16", True)
    c[1][:] = torch.randint(120, 132, c[1].shape, generator=g, dtype=torch.uint8).cuda()
    c[1][::3, :, 1] = 87
    c[1][1::3, :, 1] = 167
    tables = S.make_tables(g, ctx, B, 9, NB)
    q = torch.randn(len(ctx), H * G, D, generator=g)
    q[:, 1] *= 1e-38
    q[:, 2] *= 2.0 ** -120
    q[:, 3] = 0
    q[:, 4] *= 1e30
    q[:, 5, 1:] *= 1e-10
    q = q.bfloat16()
    sel = random_lists(g, ctx, H, B, top_k)
    for scale in (1e-31, 3e-44):
        out = torch.full(q.shape, math.nan, dtype=torch.float32, device="cuda")
        pa.pa_decode_sparse(out, q.cuda(), c[0], tables.cuda(), i32(ctx), sel.cuda(), scale=scale, scales=c[1])
        want, tol = want_sparse(q, S.host_cache(c), tables, ctx, sel, B, float(np.float32(scale)), "bf16", True)
        R.close(out, want, tol, f"scale {scale}")


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("N, top_k", [(2, 60), (30, 60), (4, 300)])
def test_waits_that_run_out_flag_and_leave_the_gpu_usable(N, top_k, quant):
    """A limit of 1 ns on every wait: the call returns with the flag (short lists join over clusters, long ones by a
    second kernel), and the next one gives the bits of one before."""
    st = Step(14, [5000] * N, 4, 4, 128, 16, "bf16", quant, top_k)
    b = st.buffers()
    sel, out = (x.clone() for x in st.run(b))
    err = err_word()
    pa.pa_set_wait_limit_ns(1)
    try:
        for _ in range(3):
            pa.pa_decode_sparse(torch.empty_like(out), st.q, st.cache[0], st.tables, st.dctx, sel, workspace=b[5],
                                dev_err=err, **scales_of(st.cache))
        torch.cuda.synchronize()
    finally:
        pa.pa_set_wait_limit_ns(0)
    assert err.item() == pa.PA_DEV_ERR_TIMEOUT
    again = torch.full_like(out, math.nan)
    err.zero_()
    pa.pa_decode_sparse(again, st.q, st.cache[0], st.tables, st.dctx, sel, workspace=b[5], dev_err=err,
                        **scales_of(st.cache))
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(again, out)


@pytest.mark.parametrize("quant", [False, True])
def test_rows_that_a_timeout_leaves_out_are_not_joined(quant):
    """Forty whole rows to a CTA, none divided, in a workspace whose cuts and parts are those of no call (in range all the
    same): after waits of 1 ns every row is as it was or as it should be, never made up from the workspace."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H, G, D, B, top_k, NB = 8, 4, 128, 16, 2, 64
    N = 40 * (7 if quant else 4) * sms // H              # CTAs per SM of the two kernels
    g = torch.Generator().manual_seed(16)
    c = S.make_cache(g, NB, H, B, D, "bf16", quant)
    tables = torch.randint(0, NB, (N, 2), generator=g).to(torch.int32).cuda()
    q = torch.randn(N, H * G, D, generator=g).bfloat16().cuda()
    ctx = i32([2 * B] * N)
    sel = torch.tensor([0, 1], dtype=torch.int32, device="cuda").expand(N, H, 2).contiguous()
    ws = torch.zeros(pa.pa_decode_sparse_workspace_bytes(N, H * G, H, D, B, top_k), dtype=torch.uint8, device="cuda")
    err = err_word()
    clean = torch.full(q.shape, math.nan, device="cuda")
    pa.pa_decode_sparse(clean, q, c[0], tables, ctx, sel, workspace=ws, dev_err=err, **scales_of(c))
    assert err.item() == 0 and not clean.isnan().any()
    left = 0
    for _ in range(3):
        ws[: 8 * N * H].fill_(0)                         # cuts (0, 0)
        ws[8 * N * H:].view(torch.float32).fill_(1.0)
        out = torch.full_like(clean, 9.0)
        pa.pa_set_wait_limit_ns(1)
        try:
            pa.pa_decode_sparse(out, q, c[0], tables, ctx, sel, workspace=ws, dev_err=err, **scales_of(c))
            torch.cuda.synchronize()
        finally:
            pa.pa_set_wait_limit_ns(0)
        untouched, right = (out == 9.0).all(-1), (out == clean).all(-1)
        assert (untouched | right).all()
        left += int(untouched.sum())
    assert left > 0 and err.item() == pa.PA_DEV_ERR_TIMEOUT


def test_tensors_of_another_place_are_refused():
    st = Step(15, [100, 50], 2, 2, 64, 16, "f16", False, 4)
    box, by, sel, out, ws1, ws2 = st.buffers()
    args = (sel, st.q, box, by, st.tables, st.dctx, 100, 16)
    for i in range(6):
        with pytest.raises(pa.PAError):
            pa.pa_select_blocks(*[x.cpu() if j == i else x for j, x in enumerate(args)])
    args = (out, st.q, st.cache[0], st.tables, st.dctx, sel)
    for i in range(6):
        with pytest.raises(pa.PAError):
            pa.pa_decode_sparse(*[x.cpu() if j == i else x for j, x in enumerate(args)])
    with pytest.raises(pa.PAError):
        pa.pa_select_blocks(sel.transpose(0, 1).contiguous().transpose(0, 1), st.q, box, by, st.tables, st.dctx, 100, 16)
    with pytest.raises(pa.PAError):
        pa.pa_select_blocks(sel.long(), st.q, box, by, st.tables, st.dctx, 100, 16)
    with pytest.raises(pa.PAError):
        pa.pa_decode_sparse(out.half().float()[:, :, ::2], st.q, st.cache[0], st.tables, st.dctx, sel)
    with pytest.raises(pa.PAError, match="workspace"):
        pa.pa_decode_sparse(out, st.q, st.cache[0], st.tables, st.dctx, sel, workspace=ws2[:16])
    with pytest.raises(pa.PAError, match="workspace"):
        pa.pa_select_blocks(sel, st.q, box, by, st.tables, st.dctx, 100, 16, workspace=ws1[:16])


_FIRST = """
import torch
import paged_kv_cache_302_gb300 as pa
pool = torch.randn(40, 16, 2, 2, 64, device="cuda").half()
tab = torch.randperm(40, device="cuda").int().view(1, 40)
ctx = torch.tensor([630], dtype=torch.int32, device="cuda")
q = torch.randn(1, 8, 64, device="cuda").half()
box = torch.zeros(40, 2, 2, 64, dtype=torch.int8, device="cuda")
by = torch.zeros(40, 2, dtype=torch.uint8, device="cuda")
sel = torch.zeros(1, 2, 9, dtype=torch.int32, device="cuda")
out, ref = torch.zeros_like(q), torch.zeros_like(q)
ks = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
keep, base = torch.arange(300, 600, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
def step(o):
    pa.pa_summarize_blocks(box, by, pool, tab, ctx, 630)
    pa.pa_select_blocks(sel, q, box, by, tab, ctx, 640, 16)
    pa.pa_decode_sparse(o, q, pool, tab, ctx, sel)
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.graph(g, stream=s):
    step(out)
    pa.pa_compact_tokens(pool, tab, ctx, base, keep, ks)
before = pool.clone()
g.replay()
torch.cuda.synchronize()
assert not torch.equal(pool, before)
pool.copy_(before)
step(ref)
assert torch.equal(out, ref) and out.abs().max() > 0
"""


def test_calls_captured_before_any_other():
    """A process whose first calls are captured into a graph."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
