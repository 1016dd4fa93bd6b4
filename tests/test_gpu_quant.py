"""The quantised cache on the GPU: the quantising write and the read bit for bit, decode attention element by element
against a 64-bit form, with poisoned memory wherever a call has no business."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _quant_ref as R
import paged_kv_cache_302_gb300 as pa

pytestmark = pytest.mark.gpu
DT = R.TORCH_DT


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def empty_cache(NB, H, B, D, fill=0x7F):
    """A cache of NaN rows with scale bytes no write produces."""
    qp = torch.full((NB, H, 2, B, D), fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    return qp, torch.full((NB, H, 2, B), 0xFF, dtype=torch.uint8, device="cuda")


def bits(qp):
    return qp.view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------------------------------------ write and read

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T, H, D, B", [(1, 1, 64, 8), (5, 2, 64, 16), (33, 3, 128, 8), (257, 8, 128, 16),
                                         (1000, 5, 64, 32), (2001, 8, 128, 32), (40, 40, 128, 16)])
def test_write_bit_exact(dtype, T, H, D, B):
    g = torch.Generator().manual_seed(T * 7 + D)
    k, v = (R.rows_like_a_model(g, (T, H, D), DT[dtype]) for _ in range(2))
    NB = -(-T // B) + 3
    slots = torch.randperm(NB * B, generator=g)[:T]
    slots[::7] = -1                                  # padding
    qp, sc = empty_cache(NB, H, B, D)
    want_q, want_s = bits(qp).copy(), sc.cpu().numpy().copy()
    err = err_word()
    pa.pa_reshape_and_cache_quant(k.cuda(), v.cuda(), qp, sc, slots.cuda(), dev_err=err)
    for i in range(T):
        s = int(slots[i])
        if s >= 0:
            for w, x in enumerate((k, v)):
                q, e = R.quantise(R.to64(x[i]))
                want_q[s // B, :, w, s % B], want_s[s // B, :, w, s % B] = q, e
    assert np.array_equal(bits(qp), want_q) and np.array_equal(sc.cpu().numpy(), want_s) and err.item() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_write_of_special_rows(dtype):
    """Zeros, a single tiny element, the type's extremes, magnitudes on both sides of 448 2^e, ties of the e4m3 grid,
    infinities and NaN."""
    D, fi = 64, torch.finfo(DT[dtype])
    rows = [torch.zeros(D)]
    for x in (fi.tiny, fi.smallest_normal, fi.max, -fi.max, 448.0, 449.0, 450.0, 447.0, 224.0, 225.0, 896.0, 2.0 ** -30):
        r = torch.zeros(D)
        r[3] = x
        rows.append(r)
    ties = torch.from_numpy((R._GRID[1:] + R._GRID[:-1]) / 2).float()
    rows += [torch.cat([ties[i: i + D - 1], torch.tensor([448.0])]) for i in range(0, len(ties) - D, D - 1)]
    for x in (math.inf, -math.inf, math.nan):
        r = torch.linspace(-3, 3, D)
        r[5] = x
        rows.append(r)
    rows.append(torch.full((D,), math.nan))
    x = torch.stack(rows).to(DT[dtype])[:, None]
    T = x.shape[0]
    qp, sc = empty_cache(-(-T // 8), 1, 8, D)
    pa.pa_reshape_and_cache_quant(x.cuda(), x.flip(0).cuda(), qp, sc, torch.arange(T).cuda())
    for w, src in enumerate((x, x.flip(0))):
        q, e = R.quantise(R.to64(src[:, 0]))
        got = bits(qp)[:, 0, w].reshape(-1, D)[:T]
        nan = np.isnan(R.to64(src[:, 0]))
        assert ((got & 0x7F) == 0x7F)[nan].all()     # a NaN of either sign
        assert np.array_equal(got[~nan], q[~nan])
        assert np.array_equal(sc.cpu().numpy()[:, 0, w].reshape(-1)[:T], e)


def test_write_flags_slots_past_the_pool_and_touches_nothing_else():
    qp, sc = empty_cache(2, 2, 8, 64)
    k = torch.ones(4, 2, 64, dtype=torch.float16, device="cuda")
    err = err_word()
    pa.pa_reshape_and_cache_quant(k, k, qp, sc, torch.tensor([16, -5, 3, 1 << 40]).cuda(), dev_err=err)
    assert err.item() == pa.PA_DEV_ERR_SLOT
    b = bits(qp)
    assert (b[0, :, :, 3] != 0x7F).all()
    b[0, :, :, 3] = 0x7F
    assert (b == 0x7F).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n, H, D, B", [(1, 1, 64, 8), (3, 3, 128, 16), (17, 8, 128, 32), (40, 5, 64, 16)])
def test_read_bit_exact(dtype, n, H, D, B):
    """Every pattern and exponent, NaN and out-of-range scale bytes among them."""
    g = torch.Generator().manual_seed(n + H)
    NS, ND = n + 5, n + 2
    qp = torch.randint(0, 256, (NS, H, 2, B, D), generator=g, dtype=torch.uint8)
    sc = torch.randint(0, 256, (NS, H, 2, B), generator=g, dtype=torch.uint8)
    sc[::2] = torch.randint(120, 132, sc[::2].shape, generator=g, dtype=torch.uint8)
    src, dst = torch.randperm(NS, generator=g)[:n], torch.randperm(ND, generator=g)[:n]
    pool = torch.full((ND, B, 2, H, D), 7.0, dtype=DT[dtype], device="cuda")
    want = torch.full(pool.shape, 7.0, dtype=torch.float64).numpy()
    x = R.values(qp.numpy(), sc.numpy())
    fi = torch.finfo(DT[dtype]).max
    for a, b in zip(src.tolist(), dst.tolist()):
        want[b] = np.clip(x[a], -fi, fi).transpose(2, 1, 0, 3)
    err = err_word()
    pa.pa_dequant_blocks(pool, qp.cuda().view(torch.float8_e4m3fn), sc.cuda(), torch.stack([src, dst], 1).cuda(),
                         dev_err=err)
    want = torch.from_numpy(want).to(DT[dtype])
    assert torch.equal(torch.nan_to_num(pool.cpu(), nan=123.0), torch.nan_to_num(want, nan=123.0))
    assert err.item() == 0


def test_read_flags_pairs_outside_the_pools():
    qp, sc = empty_cache(3, 1, 8, 64, fill=0x38)
    sc.fill_(127)
    pool = torch.zeros(2, 8, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    err = err_word()
    pa.pa_dequant_blocks(pool, qp, sc, torch.tensor([[3, 0], [0, 2], [-1, 0], [2, 1], [0, 1 << 40]]).cuda(), dev_err=err)
    assert err.item() == pa.PA_DEV_ERR_BLOCK
    assert (pool[0] == 0).all() and (pool[1] == 1).all()


def test_copy_and_swap_move_quantised_blocks():
    g = torch.Generator().manual_seed(3)
    qp = torch.randint(0, 256, (12, 3, 2, 16, 64), generator=g, dtype=torch.uint8).cuda()
    sc = torch.randint(0, 256, (12, 3, 2, 16), generator=g, dtype=torch.uint8).cuda()
    q0, s0 = qp.clone(), sc.clone()
    pairs = torch.tensor([[0, 5], [7, 2], [0, 9]]).cuda()
    for x in (qp.view(torch.float8_e4m3fn), sc):
        pa.pa_copy_blocks(x, pairs)
    for a, b in pairs.tolist():
        q0[b], s0[b] = q0[a], s0[a]
    assert torch.equal(qp, q0) and torch.equal(sc, s0)
    hq, hs = (torch.zeros((4,) + x.shape[1:], dtype=torch.uint8).pin_memory() for x in (qp, sc))
    out = torch.tensor([[5, 1], [11, 3]])
    for h, x in ((hq, qp), (hs, sc)):
        pa.pa_swap_blocks(h, x, out.cuda())
    torch.cuda.synchronize()
    assert torch.equal(hq[1], qp[5].cpu()) and torch.equal(hs[3], sc[11].cpu())
    qp.zero_()
    pa.pa_swap_blocks(qp, hq, torch.tensor([[1, 5]]).cuda())
    torch.cuda.synchronize()
    assert torch.equal(qp[5].cpu(), hq[1]) and int(qp.sum()) == int(hq[1].sum())


# ------------------------------------------------------------------------------------------------ decode

class Cache:
    """A quantised cache of random rows for given context lengths: table order shuffled, unused slots NaN with scale
    bytes no write produces, unused table entries far outside the pool."""

    def __init__(self, seed, ctx, H, D, B, dtype, spare=3, quant=True):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.H, self.D, self.B, self.dtype = list(ctx), H, D, B, DT[dtype]
        N, MB = len(ctx), max(1, max(-(-c // B) for c in ctx))
        used = [-(-c // B) for c in ctx]
        NB = sum(used) + spare
        ids = torch.randperm(NB, generator=g).tolist()
        self.tables = torch.full((N, MB), 1 << 30, dtype=torch.int32)
        slots, at = [], 0
        for s in range(N):
            t = ids[at: at + used[s]]
            at += used[s]
            self.tables[s, : used[s]] = torch.tensor(t, dtype=torch.int32)
            slots += [t[p // B] * B + p % B for p in range(ctx[s])]
        T = len(slots)
        self.k, self.v = (R.rows_like_a_model(g, (T, H, D), self.dtype) for _ in range(2))
        self.start = np.concatenate([[0], np.cumsum(ctx)])
        self.slots = torch.tensor(slots, dtype=torch.int64)
        self.MB, self.NB = MB, NB
        if quant:
            self.qp, self.sc = empty_cache(NB, H, B, D)
            pa.pa_reshape_and_cache_quant(self.k.cuda(), self.v.cuda(), self.qp, self.sc, self.slots.cuda())
        else:
            self.pool = torch.full((NB, B, 2, H, D), math.nan, dtype=self.dtype, device="cuda")
            pa.pa_reshape_and_cache(self.k.cuda(), self.v.cuda(), self.pool, self.slots.cuda())
        self.quant = quant
        self.dtab, self.dctx = self.tables.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda()

    def rows(self, s, h):
        """K and V [ctx, D] in float64 as the cache holds them, and V's exponents."""
        a, b = self.start[s], self.start[s + 1]
        out = []
        for x in (self.k, self.v):
            x = R.to64(x[a:b, h])
            if self.quant:
                q, e = R.quantise(x)
                out += [R.values(q, e), e.astype(np.float64) - 127]
            else:
                out += [x, np.zeros(b - a)]
        return out[0], out[2], out[3]


def check_decode(c: Cache, G, seed=0, scale=None, pt=0, out_dtype=torch.float32, q=None):
    N, H_q = len(c.ctx), G * c.H
    if q is None:
        q = torch.randn(N, H_q, c.D, generator=torch.Generator().manual_seed(seed)).to(c.dtype)
    out = torch.full((N, H_q, c.D), math.nan, dtype=out_dtype, device="cuda")
    err = err_word()
    pa.pa_decode_quant(out, q.cuda(), c.qp, c.sc, c.dtab, c.dctx, max(c.ctx), scale=scale, partition_tokens=pt,
                       dev_err=err)
    assert err.item() == 0
    sc = 1 / math.sqrt(c.D) if scale is None else scale
    for s in range(N):
        for h in range(c.H):
            k, v, ev = c.rows(s, h)
            want, tol = R.attend(R.to64(q[s, h * G: (h + 1) * G]), k, v, ev, np.ones((G, len(k)), bool), sc, True, True)
            R.close(out[s, h * G: (h + 1) * G], want, tol, f"sequence {s} (ctx {c.ctx[s]}), head {h}")
    return out


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D, B", [(64, 8), (64, 32), (128, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("G", [1, 4, 7, 8])
def test_decode_against_64_bits(dtype, D, B, G):
    ctx = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 129, 511, 512, 513]
    check_decode(Cache(G * D + B, ctx, 2, D, B, dtype), G)


@pytest.mark.parametrize("pt", [0, -1, 32, 96, 512])
def test_decode_partitions(pt):
    check_decode(Cache(5, [1, 40, 511, 512, 1025, 3000], 3, 128, 16, "bf16"), 5, pt=pt)
    check_decode(Cache(6, [1, 40, 511, 512, 1025, 3000], 1, 64, 8, "f16"), 2, pt=pt)


@pytest.mark.parametrize("dtype, out", [("f16", torch.float16), ("bf16", torch.bfloat16)])
def test_decode_16_bit_outputs(dtype, out):
    check_decode(Cache(8, [3, 77, 600, 1400], 8, 128, 16, dtype), 4, out_dtype=out)


def test_decode_random_shapes():
    r = np.random.default_rng(12)
    for i in range(24):
        N, H = int(r.integers(1, 9)), int(r.choice([1, 2, 3, 5, 8]))
        D, B = int(r.choice([64, 128])), int(r.choice([8, 16, 32]))
        ctx = r.integers(1, int(r.choice([30, 300, 2500])), size=N).tolist()
        check_decode(Cache(100 + i, ctx, H, D, B, str(r.choice(["f16", "bf16"]))), int(r.integers(1, 9)), seed=i,
                     pt=int(r.choice([0, -1, 64, 160])), scale=float(r.choice([0.05, 0.125, 1.0])))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_decode_values_of_very_different_size(dtype):
    """Tokens whose V differ by 2^40 (bf16) or 2^20, queries of very different rows, the largest V on an unlikely
    token: the running reference follows score and size together."""
    c = Cache(9, [200, 700], 2, 128, 16, dtype)
    span = 40 if dtype == "bf16" else 18
    g = torch.Generator().manual_seed(1)
    size = torch.exp2(torch.randint(-span // 2, span // 2 - 4, (c.v.shape[0], 2, 1), generator=g).float())
    c.v = (torch.randn(c.v.shape, generator=g) * size).clamp(-6e4, 6e4).to(c.dtype)
    c.k = (torch.randn(c.k.shape, generator=g) * 3).to(c.dtype)
    pa.pa_reshape_and_cache_quant(c.k.cuda(), c.v.cuda(), c.qp, c.sc, c.slots.cuda())
    q = torch.randn(2, 8, 128, generator=g) * torch.exp2(torch.arange(8.0) - 4)[:, None]
    check_decode(c, 4, q=q.to(c.dtype))


def test_decode_queries_of_extreme_size():
    """bf16 queries far outside fp16's range, one element dominating, and a zero query."""
    c = Cache(10, [50, 300], 1, 64, 8, "bf16")
    q = torch.randn(2, 3, 64, generator=torch.Generator().manual_seed(2))
    q[0, 0] *= 1e9
    q[0, 1] *= 1e-9
    q[0, 2] = 0
    q[1, 0, 5] = 3e4
    q[1, 1] *= 1e-30
    out = check_decode(c, 3, q=q.to(torch.bfloat16), scale=1e-9)
    assert out.isfinite().all()


def test_decode_flags_and_leaves_rows_of_bad_lengths():
    c = Cache(11, [20, 30, 40], 2, 64, 8, "f16")
    q = torch.randn(3, 4, 64).half().cuda()
    ref = torch.empty(3, 4, 64, device="cuda")
    pa.pa_decode_quant(ref, q, c.qp, c.sc, c.dtab, c.dctx, 40)
    for bad in (0, -3, 41, 1 << 30):
        ctx = c.dctx.clone()
        ctx[1] = bad
        out = torch.full_like(ref, 7.0)
        err = err_word()
        pa.pa_decode_quant(out, q, c.qp, c.sc, c.dtab, ctx, 40, dev_err=err)
        assert err.item() == pa.PA_DEV_ERR_CTX
        assert (out[1] == 7).all() and torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])


def test_decode_flags_bad_blocks_and_reads_zeros_there():
    c = Cache(12, [24, 64], 2, 128, 8, "bf16")
    q = torch.randn(2, 4, 128).bfloat16().cuda()
    ref, out = (torch.empty(2, 4, 128, device="cuda") for _ in range(2))
    pa.pa_decode_quant(ref, q, c.qp, c.sc, c.dtab, c.dctx, 64)
    for bad in (c.NB, -1, 1 << 30):
        tab = c.dtab.clone()
        tab[0, 1] = bad
        err = err_word()
        pa.pa_decode_quant(out, q, c.qp, c.sc, tab, c.dctx, 64, dev_err=err)
        assert err.item() == pa.PA_DEV_ERR_BLOCK and out.isfinite().all() and torch.equal(out[1], ref[1])


def test_decode_into_pinned_memory_graph_replay_and_streams():
    c = Cache(13, [700, 33, 1500], 4, 128, 16, "bf16")
    q = torch.randn(3, 16, 128).bfloat16().cuda()
    ref = torch.empty(3, 16, 128, device="cuda")
    ws = [torch.empty(pa.pa_decode_workspace_bytes(3, 16, 4, 128, 1500), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    pa.pa_decode_quant(ref, q, c.qp, c.sc, c.dtab, c.dctx, 1500, workspace=ws[0])
    host = torch.empty(3, 16, 128).pin_memory()
    pa.pa_decode_quant(host, q, c.qp, c.sc, c.dtab, c.dctx, 1500, workspace=ws[0])
    torch.cuda.synchronize()
    assert torch.equal(host, ref.cpu())
    # two captured graphs with workspaces of their own, replayed side by side on streams of their own
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    for st, w in zip(streams, ws):
        o = torch.zeros_like(ref)
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            pa.pa_decode_quant(o, q, c.qp, c.sc, c.dtab, c.dctx, 1500, workspace=w)
        graphs.append(g)
        outs.append(o)
    for _ in range(5):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    # the graph reads the lengths on the device anew
    c.dctx.copy_(torch.tensor([650, 20, 1400], dtype=torch.int32))
    pa.pa_decode_quant(ref, q, c.qp, c.sc, c.dtab, c.dctx, 1500, workspace=ws[1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref)


def test_decode_blocks_behind_32_bit_offsets():
    """A pool of 4.9 GB: the sequence's blocks lie past 2^31 and 2^32 bytes."""
    H, D, B, NB = 8, 128, 16, 150_000
    qp = torch.zeros(NB, H, 2, B, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc = torch.zeros(NB, H, 2, B, dtype=torch.uint8, device="cuda")
    ids = [66_000, NB - 1, 131_073, 5, 140_000]
    g = torch.Generator().manual_seed(4)
    k, v = (R.rows_like_a_model(g, (70, H, D), torch.bfloat16) for _ in range(2))
    slots = torch.tensor([ids[p // B] * B + p % B for p in range(70)])
    pa.pa_reshape_and_cache_quant(k.cuda(), v.cuda(), qp, sc, slots.cuda())
    q = torch.randn(1, 16, D, generator=g).bfloat16()
    out = torch.empty(1, 16, D, device="cuda")
    pa.pa_decode_quant(out, q.cuda(), qp, sc, torch.tensor([ids], dtype=torch.int32).cuda(),
                       torch.tensor([70], dtype=torch.int32).cuda(), 70)
    back = torch.zeros(5, B, 2, H, D, dtype=torch.bfloat16, device="cuda")
    pa.pa_dequant_blocks(back, qp, sc, torch.tensor([[b, i] for i, b in enumerate(ids)]).cuda())
    for h in range(H):
        qk, ek = R.quantise(R.to64(k[:, h]))
        qv, ev = R.quantise(R.to64(v[:, h]))
        want, tol = R.attend(R.to64(q[0, 2 * h: 2 * h + 2]), R.values(qk, ek), R.values(qv, ev), ev - 127.0,
                             np.ones((2, 70), bool), 1 / math.sqrt(D), True, True)
        R.close(out[0, 2 * h: 2 * h + 2], want, tol, f"head {h}")
        got = back[:, :, 1, h].reshape(-1, D)[:70].double().cpu().numpy()
        assert np.array_equal(got, R.values(qv, ev))


def test_a_serving_run_on_the_quantised_cache():
    """The calls together, as a server makes them: prompts quantised through the allocator's slots, a fork with a
    copy-on-write block, decode steps that write their token and attend, a chunk of prefill over the restored prefix."""
    H, G, D, B, NB = 2, 4, 64, 16, 64
    g = torch.Generator().manual_seed(20)
    al = pa.BlockAllocator(NB, B)
    qp, sc = empty_cache(NB, H, B, D)
    hist = {}

    def write(seqs, counts):
        slots, pairs, _ = al.append_batch(seqs, counts, table_updates=True)
        if len(pairs):
            for x in (qp, sc):
                pa.pa_copy_blocks(x, torch.from_numpy(np.ascontiguousarray(pairs)).cuda())
        k, v = (R.rows_like_a_model(g, (len(slots), H, D), torch.bfloat16) for _ in range(2))
        pa.pa_reshape_and_cache_quant(k.cuda(), v.cuda(), qp, sc, torch.from_numpy(slots.copy()).cuda())
        at = 0
        for s, n in zip(seqs, counts):
            hist[s] = [torch.cat([a, b[at: at + n]]) for a, b in zip(hist[s], (k, v))]
            at += n

    for s, n in ((0, 37), (1, 16)):
        al.add_seq(s)
        hist[s] = [torch.zeros(0, H, D, dtype=torch.bfloat16)] * 2
        write([s], [n])
    al.fork(0, 2)
    hist[2] = list(hist[0])
    for step in range(3):
        write([0, 1, 2], [1, 1, 1])
        tab, ctx = al.block_tables([0, 1, 2], 8)
        q = torch.randn(3, G * H, D, generator=g).bfloat16()
        out = torch.empty(3, G * H, D, device="cuda")
        pa.pa_decode_quant(out, q.cuda(), qp, sc, torch.from_numpy(tab).cuda(), torch.from_numpy(ctx).cuda(), 64)
        for s in range(3):
            for h in range(H):
                (qk, ek), (qv, ev) = (R.quantise(R.to64(x[:, h])) for x in hist[s])
                want, tol = R.attend(R.to64(q[s, h * G: h * G + G]), R.values(qk, ek), R.values(qv, ev), ev - 127.0,
                                     np.ones((G, len(qk)), bool), 1 / math.sqrt(D), True, True)
                R.close(out[s, h * G: h * G + G], want, tol, f"step {step}, sequence {s}, head {h}")
    # a chunk of prefill over sequence 2: its prefix restored to 16 bits, the chunk written as it is
    n, chunk = al.seq_len(2), 21
    table = al.block_table(2)
    own = -(-(n + chunk) // B)
    pool = torch.zeros(own, B, 2, H, D, dtype=torch.bfloat16, device="cuda")
    pa.pa_dequant_blocks(pool, qp, sc, torch.tensor([[int(b), i] for i, b in enumerate(table)]).cuda())
    k, v = (R.rows_like_a_model(g, (chunk, H, D), torch.bfloat16) for _ in range(2))
    pa.pa_reshape_and_cache(k.cuda(), v.cuda(), pool, torch.arange(n, n + chunk).cuda())
    q = torch.randn(chunk, G * H, D, generator=g).bfloat16()
    out = torch.empty(chunk, G * H, D, device="cuda")
    pa.pa_prefill(out, q.cuda(), pool, torch.arange(own, dtype=torch.int32).view(1, -1).cuda(),
                  torch.tensor([n + chunk], dtype=torch.int32).cuda(), torch.tensor([0, chunk], dtype=torch.int32).cuda(),
                  chunk)
    for h in range(H):
        (qk, ek), (qv, ev) = (R.quantise(R.to64(x[:, h])) for x in hist[2])
        kk, vv = (np.concatenate([a, R.to64(b[:, h])]) for a, b in ((R.values(qk, ek), k), (R.values(qv, ev), v)))
        see = np.arange(n + chunk)[None] <= n + np.arange(chunk)[:, None]
        for j in range(G):
            want, tol = R.attend(R.to64(q[:, h * G + j]), kk, vv, np.zeros(n + chunk), see, 1 / math.sqrt(D), False, True)
            R.close(out[:, h * G + j], want, tol, f"prefill head {h}")


class short_waits:
    """Context in which every wait inside newly launched kernels gives up after 1 ns."""

    def __enter__(self):
        pa.pa_set_wait_limit_ns(1)

    def __exit__(self, *exc):
        pa.pa_set_wait_limit_ns(0)


@pytest.mark.parametrize("pt", [0, -1])
def test_decode_timeout_exit_flags_returns_and_leaves_nothing_behind(pt):
    c = Cache(70, [700, 33, 1500, 2400] * 8, 4, 128, 16, "bf16")
    q = torch.randn(32, 16, 128).bfloat16().cuda()
    ws = torch.empty(pa.pa_decode_workspace_bytes(32, 16, 4, 128, 2400, pt), dtype=torch.uint8, device="cuda")
    ref, out, err = torch.empty(32, 16, 128, device="cuda"), torch.empty(32, 16, 128, device="cuda"), err_word()

    def run(o):
        pa.pa_decode_quant(o, q, c.qp, c.sc, c.dtab, c.dctx, 2400, partition_tokens=pt, workspace=ws, dev_err=err)

    run(ref)
    torch.cuda.synchronize()
    with short_waits():
        for _ in range(3):
            run(out)
        torch.cuda.synchronize()
    assert err.item() & pa.PA_DEV_ERR_TIMEOUT
    err.zero_()
    run(out)
    assert err.item() == 0 and torch.equal(out, ref)


def test_decode_is_the_same_every_time_and_with_the_least_workspace():
    """Equal calls give equal bits; a workspace that holds the longest partitions only still serves."""
    c = Cache(71, [2100, 600, 5, 513], 2, 128, 16, "f16")
    q = torch.randn(4, 8, 128).half().cuda()
    args = (q, c.qp, c.sc, c.dtab, c.dctx, 2100)
    a, b = (torch.empty(4, 8, 128, device="cuda") for _ in range(2))
    pa.pa_decode_quant(a, *args)
    for _ in range(10):
        pa.pa_decode_quant(b, *args)
        assert torch.equal(a, b)
    least = pa.pa_decode_workspace_bytes(4, 8, 2, 128, 2100, 512)
    pa.pa_decode_quant(b, *args, partition_tokens=512)
    ws = torch.full((least + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    pa.pa_decode_quant(a, *args, partition_tokens=512, workspace=ws[:least])
    assert torch.equal(a, b) and (ws[least:] == 0xA5).all()


def test_decode_of_sequences_that_share_blocks():
    """Eight sequences on the same prefix blocks, and the same sequence twice."""
    c = Cache(72, [300, 300], 2, 64, 16, "bf16")
    tab = c.dtab[:1].repeat(8, 1)
    q = torch.randn(1, 8, 64).bfloat16().cuda().repeat(8, 1, 1)
    out = torch.empty(8, 8, 64, device="cuda")
    pa.pa_decode_quant(out, q, c.qp, c.sc, tab, c.dctx[:1].repeat(8), 300)
    one = torch.empty(1, 8, 64, device="cuda")
    pa.pa_decode_quant(one, q[:1], c.qp, c.sc, tab[:1], c.dctx[:1], 300)
    assert torch.equal(out, out[:1].repeat(8, 1, 1))
    for h in range(2):
        k, v, ev = c.rows(0, h)
        want, tol = R.attend(R.to64(q[0, 4 * h: 4 * h + 4]), k, v, ev, np.ones((4, 300), bool), 1 / 8, True, True)
        for o in (out, one):                         # partitions may differ in length
            R.close(o[0, 4 * h: 4 * h + 4], want, tol, f"head {h}")


def test_read_into_a_pool_that_is_16_byte_aligned_only():
    g = torch.Generator().manual_seed(5)
    qp = torch.randint(0, 120, (4, 2, 2, 8, 64), generator=g, dtype=torch.uint8).cuda()
    sc = torch.randint(120, 132, (4, 2, 2, 8), generator=g, dtype=torch.uint8).cuda()
    pairs = torch.tensor([[3, 0], [1, 2]]).cuda()
    n = 3 * 8 * 2 * 2 * 64
    base = torch.zeros(n + 16, dtype=torch.float16, device="cuda")
    odd, even = base[8: 8 + n].view(3, 8, 2, 2, 64), torch.zeros(3, 8, 2, 2, 64, dtype=torch.float16, device="cuda")
    assert odd.data_ptr() % 32 == 16
    pa.pa_dequant_blocks(odd, qp, sc, pairs)
    pa.pa_dequant_blocks(even, qp, sc, pairs)
    assert torch.equal(odd, even) and even.abs().sum() > 0 and (base[:8] == 0).all() and (base[8 + n:] == 0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_decode_workspace_and_output_that_are_16_byte_aligned_only(D):
    c = Cache(73, [2100, 600, 5, 513], 2, D, 16, "f16")
    q = torch.randn(4, 8, D, generator=torch.Generator().manual_seed(6)).half().cuda()
    need = pa.pa_decode_workspace_bytes(4, 8, 2, D, 2100)
    base = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = base[16: 16 + need]
    for dt in (torch.float32, torch.float16):
        k = 16 // torch.empty(0, dtype=dt).element_size()
        outs = torch.zeros(4 * 8 * D + 2 * k, dtype=dt, device="cuda")
        out, want = outs[k:-k].view(4, 8, D), torch.zeros(4, 8, D, dtype=dt, device="cuda")
        assert out.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
        pa.pa_decode_quant(out, q, c.qp, c.sc, c.dtab, c.dctx, 2100, workspace=ws)
        pa.pa_decode_quant(want, q, c.qp, c.sc, c.dtab, c.dctx, 2100)
        assert torch.equal(out, want) and (outs[:k] == 0).all() and (outs[-k:] == 0).all()
        assert (base[:16] == 0xA5).all() and (base[16 + need:] == 0xA5).all()


@pytest.mark.parametrize("call", ["decode_quant", "tree", "decode", "prefill"])
def test_a_workspace_made_by_a_call_on_another_stream_stays_with_that_stream(call, monkeypatch):
    """The library's own workspace of a call on a side stream does not serve the current stream's next allocation, which
    may be written while the call's kernels run.  (Nothing is written here: only the addresses are compared.)"""
    quant = call in ("decode_quant", "tree")
    c = Cache(74, [2100, 600], 2, 128, 16, "bf16", quant=quant)
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    qs, mask = torch.arange(3, dtype=torch.int32).cuda(), torch.ones(2, 1, dtype=torch.int32).cuda()

    def run(out, **kw):
        if call == "decode_quant":
            pa.pa_decode_quant(out, q, c.qp, c.sc, c.dtab, c.dctx, 2100, **kw)
        elif call == "tree":
            pa.pa_decode_tree(out, q, c.qp, c.dtab, c.dctx, qs, mask, 1, scales=c.sc, **kw)
        elif call == "decode":
            pa.pa_decode(out, q, c.pool, c.dtab, c.dctx, 2100, **kw)
        else:
            pa.pa_prefill(out, q, c.pool, c.dtab, c.dctx, qs, 1, **kw)

    ref, out = torch.empty(2, 8, 128, device="cuda"), torch.empty(2, 8, 128, device="cuda")
    run(ref)
    torch.cuda.synchronize()
    made, empty = [], torch.empty

    def recorded(*a, **kw):
        t = empty(*a, **kw)
        made.append((t.data_ptr(), t.numel()))
        return t

    side = torch.cuda.Stream()
    monkeypatch.setattr(torch, "empty", recorded)
    run(out, stream=side)
    monkeypatch.setattr(torch, "empty", empty)
    (at, size), = made
    later = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    assert all(t.data_ptr() + size <= at or at + size <= t.data_ptr() for t in later)


_NAMED = """
import torch
import paged_kv_cache_302_gb300 as pa
g = torch.Generator(device="cuda").manual_seed(1)
NB, H, B, D, ctx = 70, 2, 16, 128, 1100
qp = torch.empty(NB, H, 2, B, D, dtype=torch.uint8, device="cuda")
sc = torch.empty(NB, H, 2, B, dtype=torch.uint8, device="cuda")
k, v = (torch.randn(NB * B, H, D, generator=g, device="cuda").bfloat16() for _ in range(2))
pa.pa_reshape_and_cache_quant(k, v, qp, sc, torch.arange(NB * B, device="cuda"))
q = torch.randn(1, 8, D, generator=g, device="cuda").bfloat16()
tab, n = torch.arange(NB, dtype=torch.int32, device="cuda")[None], torch.tensor([ctx], dtype=torch.int32).cuda()
outs = {pt: pa.pa_decode_quant(torch.empty(1, 8, D, device="cuda"), q, qp, sc, tab, n, ctx, partition_tokens=pt)
        for pt in (0, 64, 160)}
assert torch.equal(outs[0], outs[160]), "the named length"
assert not torch.equal(outs[0], outs[64])         # sums joined at other places: the lengths can be told apart
"""


def test_decode_takes_the_named_partition_length():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _NAMED], env={**os.environ, "PA_DECODE_PARTITION": "160"}, cwd=root,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.skipif("PA_DECODE_PARTITION" in os.environ, reason="a named length holds whatever the workspace")
def test_decode_takes_the_longest_partitions_where_the_workspace_holds_no_others():
    """partition_tokens = 0 with a workspace from the least size on: the short partitions of a small batch where they
    fit, else those of 512 tokens, and nothing behind the workspace written; below the least size a refusal."""
    c = Cache(75, [2100, 600, 5, 513], 2, 128, 16, "f16")
    q = torch.randn(4, 8, 128, generator=torch.Generator().manual_seed(8)).half().cuda()
    args = (q, c.qp, c.sc, c.dtab, c.dctx, 2100)
    least, room = (pa.pa_decode_workspace_bytes(4, 8, 2, 128, 2100, pt) for pt in (512, 0))
    assert room == pa.pa_decode_workspace_bytes(4, 8, 2, 128, 2100, 64) > least
    long, short, out = (torch.empty(4, 8, 128, device="cuda") for _ in range(3))
    pa.pa_decode_quant(long, *args, partition_tokens=512)
    pa.pa_decode_quant(short, *args, partition_tokens=64)
    assert not torch.equal(long, short)              # sums joined at other places: the lengths can be told apart
    base = torch.empty(room + 256, dtype=torch.uint8, device="cuda")
    for size, want in ((least, long), (least + 16, long), (room - 1, long), (room, short), (room + 64, short)):
        base.fill_(0xA5)
        out.zero_()
        pa.pa_decode_quant(out, *args, workspace=base[:size])
        assert torch.equal(out, want) and (base[size:] == 0xA5).all()
    with pytest.raises(pa.PAError, match="too small"):
        pa.pa_decode_quant(out, *args, workspace=base[: least - 1])


@pytest.mark.parametrize("call", ["decode_quant", "tree"])
def test_calls_without_a_workspace_captured_on_a_forked_stream(call):
    """A graph whose call runs on a stream forked from the captured one, with the library's own workspace: replays give
    the eager call's bits, whatever the program allocates and writes in between."""
    c = Cache(76, [2100, 600], 2, 128, 16, "bf16")
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    qs, mask = torch.arange(3, dtype=torch.int32).cuda(), torch.ones(2, 1, dtype=torch.int32).cuda()

    def run(out, **kw):
        if call == "decode_quant":
            return pa.pa_decode_quant(out, q, c.qp, c.sc, c.dtab, c.dctx, 2100, **kw)
        return pa.pa_decode_tree(out, q, c.qp, c.dtab, c.dctx, qs, mask, 1, scales=c.sc, **kw)

    ref = run(torch.empty(2, 8, 128, device="cuda"))
    out = torch.zeros_like(ref)
    main, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        run(out, stream=side)
        main.wait_stream(side)
    for _ in range(3):
        torch.full((64 << 20,), 0xA5, dtype=torch.uint8, device="cuda")
        out.zero_()
        graph.replay()
        assert torch.equal(out, ref)
