"""Attention for trees of drafted tokens, over 16-bit and quantised pools, element by element against a 64-bit form."""
import math

import numpy as np
import pytest
import torch

import _quant_ref as R
import paged_kv_cache_302_gb300 as pa
from test_gpu_quant import DT, Cache, err_word, short_waits

pytestmark = pytest.mark.gpu


def random_tree(r, n, chain=0.5):
    """[n, n] bool: token i sees its ancestors and itself; the parent is an earlier token or the context."""
    see = np.zeros((n, n), bool)
    for i in range(n):
        par = i - 1 if r.random() < chain else int(r.integers(-1, i)) if i else -1
        if par >= 0:
            see[i] = see[par]
        see[i, i] = True
    return see


def pack(masks, W, extra_rows=0, junk=None):
    """Packed words [T, W] of per-sequence bool masks; bits from n_s on are set at random when `junk` is given."""
    rows = []
    for m in masks:
        n = m.shape[0]
        b = np.zeros((n, W * 32), bool) if junk is None else junk.random((n, W * 32)) < 0.5
        b[:, :n] = m
        rows.append(np.packbits(b, axis=1, bitorder="little").view(np.uint32))
    rows.append(np.zeros((extra_rows, W), np.uint32))
    return torch.from_numpy(np.concatenate(rows).view(np.int32))


def run_tree(c, q, masks, W=None, out_dtype=torch.float32, scale=None, max_q=None, extra_rows=0, junk=None, ws=None,
             err=None, out=None):
    n = [m.shape[0] for m in masks]
    qs = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32).cuda()
    W = W or max(1, -(-max(n) // 32))
    if out is None:
        out = torch.full(q.shape, 7.0, dtype=out_dtype, device="cuda")
    pa.pa_decode_tree(out, q, c.qp if c.quant else c.pool, c.dtab, c.dctx, qs,
                      pack(masks, W, extra_rows, junk).cuda(), max_q or max(n), scale=scale,
                      scales=c.sc if c.quant else None, workspace=ws, dev_err=err)
    return out


def check(c, G, masks, seed=0, out_dtype=torch.float32, scale=None, q=None, **kw):
    """Runs a tree call and compares every element; the drafts are the last tokens of each sequence of `c`."""
    T = sum(m.shape[0] for m in masks)
    if q is None:
        q = torch.randn(T + kw.get("extra_rows", 0), G * c.H, c.D,
                        generator=torch.Generator().manual_seed(seed)).to(c.dtype)
    err = err_word()
    out = run_tree(c, q.cuda(), masks, out_dtype=out_dtype, scale=scale, err=err, **kw)
    assert err.item() == 0
    compare(c, G, masks, q, out, scale)
    assert (out[T:] == 7).all()
    return out


def compare(c, G, masks, q, out, scale=None):
    sc = 1 / math.sqrt(c.D) if scale is None else scale
    fp16 = c.quant or c.dtype == torch.float16
    split = not fp16 or out.dtype == torch.float32
    at = 0
    for s, m in enumerate(masks):
        n, L = m.shape[0], c.ctx[s]
        see = np.ones((n, L), bool)
        see[:, L - n:] = m
        for h in range(c.H):
            k, v, ev = c.rows(s, h)
            unseen = ~see.any(axis=0)
            k, v = np.where(unseen[:, None], 0.0, k), np.where(unseen[:, None], 0.0, v)
            qq = R.to64(q[at: at + n, h * G: (h + 1) * G]).reshape(n * G, c.D)
            want, tol = R.attend(qq, k, v, ev, np.repeat(see, G, axis=0), sc, split, fp16)
            R.close(out[at: at + n, h * G: (h + 1) * G].reshape(n * G, c.D), want, tol,
                    f"sequence {s} (ctx {L}, draft {n}), head {h}")
        at += n


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D, B, G", [(128, 16, 4), (128, 8, 1), (128, 32, 7), (64, 16, 8), (64, 8, 3)])
def test_tree_against_64_bits(quant, dtype, D, B, G):
    r = np.random.default_rng(D + B + G)
    ctx = [1, 2, 9, 40, 127, 128, 129, 200, 255, 256, 257, 300, 511, 700]
    n = [1, 1, 9, 8, 5, 16, 3, 1, 12, 7, 2, 13, 4, 16]
    check(Cache(G * D + B, ctx, 2, D, B, dtype, quant=quant), G, [random_tree(r, i) for i in n])


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("G, n", [(1, 128), (1, 129), (4, 32), (4, 33), (8, 64), (3, 43), (40, 3), (40, 4), (128, 1),
                                  (128, 3), (100, 2), (7, 63)])
def test_tree_row_tiles(quant, G, n):
    """Query rows (drafted tokens x heads per KV head) around and above one tile of 128."""
    r = np.random.default_rng(G + n)
    c = Cache(G + n, [n + 150, n, n + 1000], 1, 128, 16, "bf16", quant=quant)
    check(c, G, [random_tree(r, n), random_tree(r, n), random_tree(r, max(1, n - 1))])


@pytest.mark.parametrize("quant", [False, True])
def test_tree_long_drafts_and_causal_masks(quant):
    """Drafts longer than a key tile, as causal chunks and as trees, masks wider than the draft with junk past it."""
    r = np.random.default_rng(4)
    for n, ctx in ((300, 300), (257, 900), (130, 131)):
        c = Cache(n, [ctx, ctx + 5], 1, 64, 16, "f16", quant=quant)
        check(c, 2, [np.tril(np.ones((n, n), bool)), random_tree(r, n - 1, 0.9)], W=12, junk=r)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_tree_16_bit_outputs(quant, dtype):
    r = np.random.default_rng(5)
    check(Cache(31, [90, 400, 1300], 4, 128, 16, dtype, quant=quant), 4, [random_tree(r, i) for i in (8, 24, 31)],
          out_dtype=DT[dtype])


@pytest.mark.parametrize("quant", [False, True])
def test_tree_long_contexts_are_split_and_joined(quant):
    r = np.random.default_rng(6)
    check(Cache(32, [9000], 2, 128, 32, "bf16", quant=quant), 4, [random_tree(r, 20)])
    check(Cache(33, [5000, 60, 3000], 3, 64, 8, "f16", quant=quant), 2,
          [random_tree(r, 70), random_tree(r, 5), random_tree(r, 33)])


@pytest.mark.parametrize("quant", [False, True])
def test_tree_random_shapes(quant):
    r = np.random.default_rng(40 + quant)
    for i in range(20):
        N, H, D, B = int(r.integers(1, 7)), int(r.choice([1, 2, 3, 5])), int(r.choice([64, 128])), int(r.choice([8, 16, 32]))
        top = int(r.choice([40, 300, 2000]))
        n = [int(x) for x in r.integers(0, int(r.choice([3, 20, 70])), size=N)]
        ctx = [max(1, x) + int(r.integers(0, top)) for x in n]
        c = Cache(200 + i, ctx, H, D, B, str(r.choice(["f16", "bf16"])), quant=quant)
        if sum(n) == 0:
            n[0] = 1
        masks = [random_tree(r, x, r.random()) if x else np.zeros((0, 0), bool) for x in n]
        for m in masks:                              # a few rows see nothing of the draft
            if m.shape[0] > 2:
                m[int(r.integers(0, m.shape[0]))] = False
        check(c, int(r.integers(1, 9)), masks, seed=i, extra_rows=int(r.integers(0, 3)),
              scale=float(r.choice([0.05, 0.125, 0.7])))


@pytest.mark.parametrize("quant", [False, True])
def test_tree_rows_that_see_nothing_are_zero(quant):
    c = Cache(50, [5, 40, 130], 2, 128, 8, "bf16", quant=quant)
    masks = [np.eye(5, dtype=bool), np.tril(np.ones((40, 40), bool)), np.tril(np.ones((130, 130), bool))]
    masks[0][2] = False
    masks[0][:, 2] = False
    masks[1][[0, 39]] = False
    masks[2][5:100] = False
    out = check(c, 3, masks)
    at = 0
    for m in masks:
        empty = torch.from_numpy(~m.any(1))
        assert (out[at: at + len(m)][empty.cuda()] == 0).all()
        at += len(m)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_tree_padding_drafts_may_hold_anything(quant, value):
    """K and V of drafted tokens that no row sees are NaN or infinite (for a quantised pool: NaN rows under scale bytes
    no write produces), beside rows that see the others."""
    c = Cache(51, [30, 200, 140], 2, 128, 16, "f16", quant=quant)
    r = np.random.default_rng(8)
    masks = [random_tree(r, 12), random_tree(r, 20), random_tree(r, 140)]
    for s, (m, pad) in enumerate(zip(masks, ([3, 11], [0, 7, 8, 9, 19], list(range(60, 90)) + [139]))):
        m[:, pad] = False
        m[pad] = False
        for j in pad:
            p = c.ctx[s] - m.shape[0] + j
            slot = int(c.slots[c.start[s] + p])
            if quant:
                c.qp.view(torch.uint8)[slot // 16, :, :, slot % 16] = 0x7F
                c.sc[slot // 16, :, :, slot % 16] = 0xFF
            else:
                c.pool[slot // 16, slot % 16] = value
    check(c, 4, masks)


@pytest.mark.parametrize("quant", [False, True])
def test_tree_of_one_token_agrees_with_decode(quant):
    """One drafted token that sees itself is a decode step."""
    c = Cache(52, [1, 17, 300, 800], 4, 128, 16, "bf16", quant=quant)
    q = torch.randn(4, 16, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    out = check(c, 4, [np.ones((1, 1), bool)] * 4, q=q)
    ref = torch.empty_like(out)
    if quant:
        pa.pa_decode_quant(ref, q.cuda(), c.qp, c.sc, c.dtab, c.dctx, 800)
    else:
        pa.pa_decode(ref, q.cuda(), c.pool, c.dtab, c.dctx, 800)
    compare(c, 4, [np.ones((1, 1), bool)] * 4, q, ref)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_tree_quantised_values_of_very_different_size(dtype):
    c = Cache(53, [260, 700], 2, 128, 16, dtype)
    span = 40 if dtype == "bf16" else 18
    g = torch.Generator().manual_seed(1)
    size = torch.exp2(torch.randint(-span // 2, span // 2 - 4, (c.v.shape[0], 2, 1), generator=g).float())
    c.v = (torch.randn(c.v.shape, generator=g) * size).clamp(-6e4, 6e4).to(c.dtype)
    pa.pa_reshape_and_cache_quant(c.k.cuda(), c.v.cuda(), c.qp, c.sc, c.slots.cuda())
    q = torch.randn(20, 8, 128, generator=g) * torch.exp2(torch.arange(8.0) - 4)[:, None]
    r = np.random.default_rng(9)
    check(c, 4, [random_tree(r, 8), random_tree(r, 12)], q=q.to(c.dtype))


def test_tree_flags_and_leaves_what_is_wrong():
    for quant in (False, True):
        c = Cache(54, [60, 70, 80], 2, 64, 16, "f16", quant=quant)
        r = np.random.default_rng(3)
        masks = [random_tree(r, 6) for _ in range(3)]
        q = torch.randn(18, 4, 64).half().cuda()
        ref = run_tree(c, q, masks)

        def call(ctx=None, qs=None, tab=None, max_q=6):
            out, err = torch.full_like(ref, 7.0), err_word()
            pa.pa_decode_tree(out, q, c.qp if quant else c.pool, c.dtab if tab is None else tab,
                              c.dctx if ctx is None else torch.tensor(ctx, dtype=torch.int32).cuda(),
                              torch.tensor([0, 6, 12, 18] if qs is None else qs, dtype=torch.int32).cuda(),
                              pack(masks, 1).cuda(), max_q, scales=c.sc if quant else None, dev_err=err)
            return out, err.item()

        for bad in (5, 0, -1, 81, 1 << 30):          # too short for its draft, too long for its table
            out, e = call(ctx=[60, bad, 80])
            assert e == pa.PA_DEV_ERR_CTX and (out[6:12] == 7).all()
            assert torch.equal(out[:6], ref[:6]) and torch.equal(out[12:], ref[12:])
        for qs in ([0, 6, 12, 19], [0, 6, 12, 1 << 30]):     # a draft that ends past q
            out, e = call(qs=qs)
            assert e == pa.PA_DEV_ERR_CTX and torch.equal(out[:12], ref[:12]) and (out[12:] == 7).all()
        out, e = call(qs=[0, 6, 3, 9])               # starts that decrease
        assert e & pa.PA_DEV_ERR_CTX and torch.equal(out[:3], ref[:3])
        out, e = call(qs=[0, 2, 12, 18])             # a draft longer than max_q_len
        assert e == pa.PA_DEV_ERR_CTX and (out[2:12] == 7).all() and torch.equal(out[12:], ref[12:])
        out, e = call(qs=[-4, 6, 12, 18])
        assert e == pa.PA_DEV_ERR_CTX and torch.equal(out[6:], ref[6:])
        for bad in (c.NB, -1, 1 << 30):
            tab = c.dtab.clone()
            tab[1, 2] = bad
            out, e = call(tab=tab)
            assert e == pa.PA_DEV_ERR_BLOCK and out.isfinite().all()
            assert torch.equal(out[:6], ref[:6]) and torch.equal(out[12:], ref[12:])


@pytest.mark.parametrize("quant", [False, True])
def test_tree_is_the_same_every_time_captured_and_beside_another_call(quant):
    c = Cache(55, [1200, 90, 2500, 31], 4, 128, 16, "bf16", quant=quant)
    r = np.random.default_rng(3)
    n = [20, 31, 9, 31]
    masks = [random_tree(r, i) for i in n]
    q = torch.randn(sum(n), 16, 128).bfloat16().cuda()
    need = pa.pa_decode_tree_workspace_bytes(4, 16, 4, 128, 31)
    ws = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ref = run_tree(c, q, masks, ws=ws[0])
    for _ in range(10):
        assert torch.equal(run_tree(c, q, masks, ws=ws[0]), ref)
    qs = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32).cuda()
    m = pack(masks, 1).cuda()
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    for st, w in zip(streams, ws):
        o = torch.zeros_like(ref)
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            pa.pa_decode_tree(o, q, c.qp if quant else c.pool, c.dtab, c.dctx, qs, m, 31,
                              scales=c.sc if quant else None, workspace=w)
        graphs.append(g)
        outs.append(o)
    for _ in range(5):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    # other lengths on the device under the same graph: the shortest and the longest the tables hold
    c.ctx = [20, 31, 2500, 31]
    c.dctx.copy_(torch.tensor(c.ctx, dtype=torch.int32))
    ref = run_tree(c, q, masks, ws=ws[1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref)


@pytest.mark.parametrize("quant", [False, True])
def test_tree_writes_nothing_outside_its_buffers(quant):
    """Every buffer the call may write lies between sentinels."""
    c = Cache(56, [500, 40], 2, 64, 8, "bf16", quant=quant)
    r = np.random.default_rng(3)
    masks = [random_tree(r, 13), random_tree(r, 40)]
    q = torch.randn(53, 6, 64).bfloat16()
    need = pa.pa_decode_tree_workspace_bytes(2, 6, 2, 64, 40)

    def fenced(nbytes):
        a = torch.full((nbytes + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        return a, a[4096: 4096 + nbytes]

    wa, w = fenced(need)
    for dt in (torch.float32, torch.bfloat16):
        oa, o = fenced(53 * 6 * 64 * (4 if dt == torch.float32 else 2))
        o = o.view(dt).view(53, 6, 64)
        run_tree(c, q.cuda(), masks, ws=w, out=o)
        compare(c, 3, masks, q, o)
        for a, size in ((oa, o.numel() * o.element_size()), (wa, need)):
            assert (a[:4096] == 0xA5).all() and (a[4096 + size:] == 0xA5).all()


def test_a_speculative_step_with_the_allocator():
    """Draft, verify, accept: the sequence is forked, the draft written into the fork (copy-on-write), verified under
    its mask, the fork freed and the accepted path appended; a decode step then sees prompt and accepted tokens."""
    H, G, D, B, NB = 2, 4, 128, 16, 40
    g = torch.Generator().manual_seed(21)
    for quant in (False, True):
        al = pa.BlockAllocator(NB, B)
        c = Cache(60, [1], H, D, B, "bf16", spare=NB - 1, quant=quant)
        stores = (c.qp, c.sc) if quant else (c.pool,)

        def write(seq, k, v):
            slots, pairs = al.append_slots(seq, k.shape[0])
            if len(pairs):
                for x in stores:
                    pa.pa_copy_blocks(x, torch.from_numpy(np.ascontiguousarray(pairs)).cuda())
            sl = torch.from_numpy(slots.copy()).cuda()
            if quant:
                pa.pa_reshape_and_cache_quant(k.cuda(), v.cuda(), c.qp, c.sc, sl)
            else:
                pa.pa_reshape_and_cache(k.cuda(), v.cuda(), c.pool, sl)

        def rows(n):
            return [R.rows_like_a_model(g, (n, H, D), torch.bfloat16) for _ in range(2)]

        al.add_seq(0)
        prompt, draft = rows(75), rows(9)
        write(0, *prompt)
        al.fork(0, 1)
        write(1, *draft)
        mask = random_tree(np.random.default_rng(2), 9, 0.4)
        tab, ctx = al.block_tables([1], 6)
        c.k, c.v = (torch.cat([a, b]) for a, b in zip(prompt, draft))
        c.start, c.ctx = np.array([0, 84]), [84]
        c.dtab, c.dctx = torch.from_numpy(tab).cuda(), torch.from_numpy(ctx).cuda()
        check(c, G, [mask])
        al.free_seq(1)
        path = np.flatnonzero(mask[8])
        write(0, draft[0][path], draft[1][path])
        tab, ctx = al.block_tables([0], 6)
        c.k, c.v = (torch.cat([a, b[path]]) for a, b in zip(prompt, draft))
        c.ctx = [75 + len(path)]
        c.start = np.array([0, c.ctx[0]])
        q = torch.randn(1, G * H, D, generator=g).bfloat16()
        out = torch.empty(1, G * H, D, device="cuda")
        args = (torch.from_numpy(tab).cuda(), torch.from_numpy(ctx).cuda(), 96)
        if quant:
            pa.pa_decode_quant(out, q.cuda(), c.qp, c.sc, *args)
        else:
            pa.pa_decode(out, q.cuda(), c.pool, *args)
        compare(c, G, [np.ones((1, 1), bool)], q, out)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_tree_timeout_exit_flags_returns_and_leaves_nothing_behind(quant, out_dtype):
    c = Cache(70, [1200, 90, 2500, 31] * 6, 4, 128, 16, "bf16", quant=quant)
    r = np.random.default_rng(3)
    masks = [random_tree(r, i) for i in (20, 31, 70, 31) * 6]
    q = torch.randn(sum(m.shape[0] for m in masks), 16, 128).bfloat16().cuda()
    ref = run_tree(c, q, masks, out_dtype=out_dtype)
    err = err_word()
    with short_waits():
        for _ in range(3):
            run_tree(c, q, masks, out_dtype=out_dtype, err=err)
        torch.cuda.synchronize()
    assert err.item() & pa.PA_DEV_ERR_TIMEOUT
    err.zero_()
    assert torch.equal(run_tree(c, q, masks, out_dtype=out_dtype, err=err), ref) and err.item() == 0


@pytest.mark.parametrize("quant", [False, True])
def test_tree_more_sequences_than_threads(quant):
    """1500 sequences, a third of them without a draft: the runs are cut over several rounds of the block's threads."""
    r = np.random.default_rng(11)
    n = [int(x) for x in r.integers(0, 3, size=1500)]
    n[700] = 9
    ctx = [x + int(r.integers(0 if x else 1, 40)) for x in n]
    ctx[1400] += 900
    check(Cache(80, ctx, 1, 64, 8, "f16", quant=quant), 2,
          [random_tree(r, x) if x else np.zeros((0, 0), bool) for x in n])


@pytest.mark.parametrize("quant", [False, True])
def test_tree_output_that_is_16_byte_aligned_only(quant):
    c = Cache(81, [60, 900], 2, 64, 16, "f16", quant=quant)
    r = np.random.default_rng(12)
    masks = [random_tree(r, 6), random_tree(r, 7)]
    q = torch.randn(13, 6, 64).half()
    for dt in (torch.float32, torch.float16):
        k = 16 // torch.empty(0, dtype=dt).element_size()
        base = torch.zeros(13 * 6 * 64 + 2 * k, dtype=dt, device="cuda")
        out = base[k:-k].view(13, 6, 64)
        assert out.data_ptr() % 32 == 16
        run_tree(c, q.cuda(), masks, out=out)
        compare(c, 3, masks, q, out)
        assert (base[:k] == 0).all() and (base[-k:] == 0).all()


@pytest.mark.parametrize("quant", [False, True])
def test_tree_blocks_behind_32_bit_offsets(quant):
    """Pools of 4.9 GB: blocks past 2^31 and 2^32 bytes, two sequences on the same prefix blocks."""
    H, G, D, B, NB = 8, 2, 128, 16, 150_000 if quant else 75_000
    ids = [NB * 2 // 5, NB - 1, NB * 9 // 10, 5, NB * 14 // 15]
    c = Cache(82, [70, 66], H, D, B, "bf16", quant=quant)
    c.tables = torch.tensor([ids, ids[:4] + [77]], dtype=torch.int32)
    c.slots = torch.tensor([t[p // B] * B + p % B for t, n in zip(c.tables.tolist(), c.ctx) for p in range(n)])
    c.k[70:134], c.v[70:134] = c.k[:64].clone(), c.v[:64].clone()
    c.dtab = c.tables.cuda()
    if quant:
        c.qp = torch.zeros(NB, H, 2, B, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        c.sc = torch.zeros(NB, H, 2, B, dtype=torch.uint8, device="cuda")
        pa.pa_reshape_and_cache_quant(c.k.cuda(), c.v.cuda(), c.qp, c.sc, c.slots.cuda())
    else:
        c.pool = torch.zeros(NB, B, 2, H, D, dtype=torch.bfloat16, device="cuda")
        pa.pa_reshape_and_cache(c.k.cuda(), c.v.cuda(), c.pool, c.slots.cuda())
    r = np.random.default_rng(13)
    check(c, G, [random_tree(r, 5), random_tree(r, 2)])


@pytest.mark.parametrize("quant", [False, True])
def test_tree_calls_of_small_heads_beside_each_other(quant):
    """D = 64: two CTAs of the 16-bit kernel fit an SM's shared memory, and the second waits for the first one's tensor
    memory.  Calls on three streams, each with a workspace of its own, give the bits they give alone."""
    r = np.random.default_rng(15)
    c = Cache(90, [3000, 700, 41, 1900] * 10, 2, 64, 16, "f16", quant=quant)
    masks = [random_tree(r, 16) for _ in c.ctx]
    q = torch.randn(16 * 40, 8, 64).half().cuda()
    ref = run_tree(c, q, masks)
    qs = torch.arange(0, 16 * 41, 16, dtype=torch.int32).cuda()
    m = pack(masks, 1).cuda()
    need = pa.pa_decode_tree_workspace_bytes(40, 8, 2, 64, 16)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.zeros_like(ref) for _ in streams]
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, o, w in zip(streams, outs, ws):
            pa.pa_decode_tree(o, q, c.qp if quant else c.pool, c.dtab, c.dctx, qs, m, 16,
                              scales=c.sc if quant else None, workspace=w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


@pytest.mark.parametrize("D, B", [(128, 16), (64, 8)])
def test_tree_quantised_queries_of_extreme_size(D, B):
    """bf16 queries far outside fp16's range under a tiny scale, over contexts that end inside a key tile: unseen keys
    count for nothing, whatever a score's factor rounds to."""
    c = Cache(57, [50, 300], 1, D, B, "bf16")
    r = np.random.default_rng(16)
    q = torch.randn(9, 3, D, generator=torch.Generator().manual_seed(2))
    q[0, 0] *= 1e9
    q[0, 1] *= 1e-9
    q[0, 2] = 0
    q[1, 0, 5] = 3e4
    q[1:3, 1] *= 1e-30
    q[5:, 2] *= 1e-36
    check(c, 3, [random_tree(r, 4), random_tree(r, 5)], q=q.to(torch.bfloat16), scale=1e-9)


@pytest.mark.parametrize("keyed", [False, True])
def test_tree_quantised_small_queries_before_key_tiles_they_do_not_see(keyed):
    """Causal drafts longer than a key tile, the default scale: later key tiles are seen by no row of the first row
    tiles, whose queries lie 2^86 and more below one; with V scales close together and far apart."""
    r = np.random.default_rng(17)
    c = Cache(58, [300, 420], 1, 64, 16, "bf16")
    if keyed:
        g = torch.Generator().manual_seed(1)
        size = torch.exp2(torch.randint(-18, 14, (c.v.shape[0], 1, 1), generator=g).float())
        c.v = (torch.randn(c.v.shape, generator=g) * size).to(c.dtype)
        pa.pa_reshape_and_cache_quant(c.k.cuda(), c.v.cuda(), c.qp, c.sc, c.slots.cuda())
    q = torch.randn(600, 2, 64, generator=torch.Generator().manual_seed(3))
    q *= torch.exp2(torch.from_numpy(r.integers(-118, -84, size=(600, 2, 1))).float())
    check(c, 2, [np.tril(np.ones((300, 300), bool))] * 2, q=q.to(torch.bfloat16))


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1e-25, 1e-38, 3e-44])
def test_tree_tiny_scales(quant, dtype, scale):
    """Scales down to fp32's subnormal numbers: nearly uniform weights of what each row sees."""
    r = np.random.default_rng(18)
    c = Cache(59, [140, 300], 2, 128, 16, dtype, quant=quant)
    check(c, 2, [np.tril(np.ones((140, 140), bool)), random_tree(r, 20)], scale=scale)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("D, B", [(128, 16), (64, 8)])
def test_tree_workspace_that_is_16_byte_aligned_only(quant, D, B):
    """A workspace cut from a larger buffer at an odd multiple of 16 bytes, sequences long enough for every unit to be
    shared by several CTAs: the same bits as with an aligned one, and nothing beside it written."""
    c = Cache(83, [6000, 130, 2500], 2, D, B, "bf16", quant=quant)
    r = np.random.default_rng(19)
    masks = [random_tree(r, 20), random_tree(r, 3), random_tree(r, 45)]
    q = torch.randn(68, 6, D, generator=torch.Generator().manual_seed(4)).bfloat16()
    need = pa.pa_decode_tree_workspace_bytes(3, 6, 2, D, 45)
    base = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        want = run_tree(c, q.cuda(), masks, out_dtype=dt)
        compare(c, 3, masks, q, want)
        for at in (16, 48, 2064):
            ws = base[at: at + need]
            assert ws.data_ptr() % 32 == 16
            assert torch.equal(run_tree(c, q.cuda(), masks, out_dtype=dt, ws=ws), want)
            assert (base[:at] == 0xA5).all() and (base[at + need:] == 0xA5).all()
            base.fill_(0xA5)
