"""Refusals of the block-sparse calls and of compaction, and the allocator's side of compaction against an independent
model, without a GPU: placeholder addresses are never dereferenced, because validation fails first."""
import ctypes

import numpy as np
import pytest
import torch

import _sparse_ref as S
import paged_kv_cache_302_gb300 as pa
from oracle.alloc_model import AllocError, AllocModel

A = [0x1000 * (i + 1) for i in range(12)]        # aligned placeholder addresses
F16, BF16, F32, E4M3 = pa.PA_F16, pa.PA_BF16, pa.PA_F32, pa.PA_E4M3
INV, UNS, OK = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED, pa.PA_OK


def summarize(box=A[0], by=A[1], pool=A[2], sc=None, kdt=BF16, tab=A[3], ctx=A[4], qs=A[5], N=2, H=2, D=128, B=16, MB=4,
              NB=8, mq=4):
    return pa.load().pa_summarize_blocks(box, by, pool, sc, kdt, tab, ctx, qs, N, H, D, B, MB, NB, mq, None, None)


def select(sel=A[0], q=A[1], qdt=BF16, box=A[2], by=A[3], tab=A[4], ctx=A[5], N=2, Hq=8, H=2, D=128, B=16, MB=4, NB=8,
           mc=64, k=2, sink=1, rec=1, ws=A[6], wsb=1 << 30):
    return pa.load().pa_select_blocks(sel, q, qdt, box, by, tab, ctx, N, Hq, H, D, B, MB, NB, mc, k, sink, rec, ws, wsb,
                                      None, None)


def decode(out=A[0], odt=F32, q=A[1], qdt=BF16, pool=A[2], sc=None, kdt=BF16, tab=A[3], ctx=A[4], sel=A[5], k=2, N=2,
           Hq=8, H=2, D=128, B=16, MB=4, NB=8, scale=0.1, ws=A[6], wsb=1 << 30):
    return pa.load().pa_decode_sparse(out, odt, q, qdt, pool, sc, kdt, tab, ctx, sel, k, N, Hq, H, D, B, MB, NB, scale, ws,
                                      wsb, None, None)


def compact(pool=A[0], sc=None, kdt=BF16, tab=A[1], ctx=A[2], base=A[3], keep=A[4], ks=A[5], N=2, T=4, H=2, D=128, B=16,
            MB=4, NB=8):
    return pa.load().pa_compact_tokens(pool, sc, kdt, tab, ctx, base, keep, ks, N, T, H, D, B, MB, NB, None, None)


@pytest.mark.parametrize("call", [summarize, select, decode, compact])
@pytest.mark.parametrize("kw, status", [
    (dict(D=96), UNS), (dict(D=256), UNS), (dict(B=4), UNS), (dict(B=64), UNS), (dict(B=0), UNS), (dict(H=0), INV),
    (dict(H=-1), INV), (dict(N=0), INV), (dict(N=65536), INV), (dict(MB=0), INV), (dict(NB=0), INV),
    (dict(NB=1 << 27), UNS), (dict(MB=1 << 27), UNS), (dict(tab=None), INV), (dict(ctx=None), INV)])
def test_calls_refuse(call, kw, status):
    assert call(**kw) == status and pa.last_error()


@pytest.mark.parametrize("call", [summarize, decode, compact])
@pytest.mark.parametrize("kw, status", [
    (dict(kdt=F32), UNS), (dict(kdt=E4M3), INV), (dict(sc=A[8]), INV), (dict(kdt=E4M3, sc=A[8] + 8), INV),
    (dict(pool=A[2] + 8), INV), (dict(pool=None), INV)])
def test_calls_refuse_caches(call, kw, status):
    assert call(**kw) == status and pa.last_error()


@pytest.mark.parametrize("call, kw, status", [
    (summarize, dict(mq=-1), INV), (summarize, dict(box=None), INV), (summarize, dict(by=None), INV),
    (summarize, dict(box=A[0] + 8), INV),
    (select, dict(qdt=F32), UNS), (select, dict(qdt=E4M3), UNS), (select, dict(Hq=7), INV), (select, dict(Hq=18), UNS),
    (select, dict(Hq=0), INV), (select, dict(mc=0), INV), (select, dict(k=0), INV), (select, dict(sink=-1), INV),
    (select, dict(rec=-1), INV), (select, dict(sink=2, rec=1), INV), (select, dict(sink=2 ** 31 - 1, rec=2 ** 31 - 1), INV),
    (select, dict(ws=None), INV), (select, dict(wsb=15), INV), (select, dict(q=A[1] + 2), INV),
    (select, dict(sel=None), INV), (select, dict(k=(1 << 28) + 1), UNS), (select, dict(box=A[2] + 8), INV), (select, dict(by=None), INV),
    (decode, dict(qdt=F32), UNS), (decode, dict(kdt=F16), UNS), (decode, dict(odt=F16), UNS), (decode, dict(Hq=7), INV),
    (decode, dict(Hq=18), UNS), (decode, dict(k=0), INV), (decode, dict(scale=0.0), INV), (decode, dict(scale=-1.0), INV),
    (decode, dict(scale=float("nan")), INV), (decode, dict(scale=float("inf")), INV), (decode, dict(ws=None), INV),
    (decode, dict(wsb=0), INV), (decode, dict(out=A[0] + 8), INV), (decode, dict(q=A[1] + 2), INV),
    (decode, dict(sel=None), INV), (decode, dict(k=(1 << 28) + 1), UNS), (decode, dict(k=1 << 28, N=4000), UNS), (compact, dict(T=-1), INV), (compact, dict(keep=None), INV),
    (compact, dict(base=None), INV), (compact, dict(ks=None), INV)])
def test_calls_refuse_their_own(call, kw, status):
    assert call(**kw) == status and pa.last_error()


def test_nothing_to_do_is_no_error():
    assert summarize(mq=0, box=None) == OK and compact(T=0, keep=None) == OK


def test_workspaces():
    assert pa.pa_select_workspace_bytes(2, 8, 1000, 16) >= 2 * 8 * 63 * 4
    assert pa.pa_decode_sparse_workspace_bytes(2, 32, 8, 128, 16, 64) > 0
    for bad in [(0, 8, 100, 16), (1, 0, 100, 16), (1, 8, 0, 16), (1, 8, 100, 4), (65536, 8, 100, 16)]:
        with pytest.raises(pa.PAError):
            pa.pa_select_workspace_bytes(*bad)
    for bad in [(0, 32, 8, 128, 16, 4), (1, 31, 8, 128, 16, 4), (1, 72, 8, 128, 16, 4), (1, 32, 8, 96, 16, 4),
                (1, 32, 8, 128, 4, 4), (1, 32, 8, 128, 16, 0)]:
        with pytest.raises(pa.PAError):
            pa.pa_decode_sparse_workspace_bytes(*bad)


def test_python_refuses_before_the_library_is_called():
    pool = torch.zeros(4, 16, 2, 2, 64, dtype=torch.float16)
    qp, sc = torch.zeros(4, 2, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 2, 16, dtype=torch.uint8)
    box, by = torch.zeros(4, 2, 2, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    tab, ctx = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    q, sel = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, 2, 3, dtype=torch.int32)
    ks = torch.zeros(3, dtype=torch.int32)

    def refused(f, *a, **kw):
        with pytest.raises(pa.PAError):
            f(*a, **kw)

    refused(pa.pa_summarize_blocks, box, by, pool, tab, ctx, 4)                       # host tensors
    refused(pa.pa_summarize_blocks, box[:3], by[:3], pool, tab, ctx, 4)               # summaries of another cache
    refused(pa.pa_summarize_blocks, box.float(), by, pool, tab, ctx, 4)
    refused(pa.pa_summarize_blocks, box, by.int(), pool, tab, ctx, 4)
    refused(pa.pa_summarize_blocks, box, by[:, :1], pool, tab, ctx, 4)
    refused(pa.pa_summarize_blocks, box, by, pool.float(), tab, ctx, 4)
    refused(pa.pa_summarize_blocks, box, by, qp, tab, ctx, 4)                         # qpool without scales
    refused(pa.pa_summarize_blocks, box, by, qp, tab, ctx, 4, scales=sc[:3])
    refused(pa.pa_summarize_blocks, box, by, pool, tab, ctx, 4, q_start=ks[:2])
    refused(pa.pa_summarize_blocks, box, by, pool, tab[:1], ctx, 4)
    refused(pa.pa_select_blocks, sel, q, box, by, tab, ctx, 8, 16)                    # host tensors
    refused(pa.pa_select_blocks, sel[:, :1], q, box, by, tab, ctx, 8, 16)
    refused(pa.pa_select_blocks, sel[0], q, box, by, tab, ctx, 8, 16)
    refused(pa.pa_select_blocks, sel, q[:1], box, by, tab, ctx, 8, 16)
    refused(pa.pa_select_blocks, sel, q[:, :, :32], box, by, tab, ctx, 8, 16)
    refused(pa.pa_select_blocks, sel, q, box, by, tab[0], ctx, 8, 16)
    refused(pa.pa_decode_sparse, q, q, pool, tab, ctx, sel)                           # host tensors
    refused(pa.pa_decode_sparse, q[:1], q, pool, tab, ctx, sel)
    refused(pa.pa_decode_sparse, q, q, pool.bfloat16(), tab, ctx, sel)
    refused(pa.pa_decode_sparse, q, q, pool, tab, ctx, sel[:, :1])
    refused(pa.pa_decode_sparse, q, q, qp, tab, ctx, sel)
    refused(pa.pa_decode_sparse, q, q, pool, tab, ctx[:1], sel)
    refused(pa.pa_compact_tokens, pool, tab, ctx, ctx, ctx, ks)                       # host tensors
    refused(pa.pa_compact_tokens, pool, tab, ctx, ctx[:1], ctx, ks)
    refused(pa.pa_compact_tokens, pool, tab, ctx, ctx, ctx, ks[:2])
    refused(pa.pa_compact_tokens, qp, tab, ctx, ctx, ctx, ks)
    refused(pa.pa_compact_tokens, pool.transpose(2, 3), tab, ctx, ctx, ctx, ks)


def test_reference_score_bounds_every_product():
    """The tests' own boxes and scores: no key's product with a query exceeds its block's score by more than the query's
    rounding, half a unit of 2^f per channel."""
    r = np.random.default_rng(0)
    for _ in range(20):
        k = r.standard_normal((16, 64)) * np.exp(r.standard_normal(64))
        q = r.standard_normal((3, 64))
        box, by = S.box(k)
        f = S.least_exponent(np.abs(q).max(axis=1), S.QUERY_TOP)
        slack = 0.5 * np.exp2(f.astype(float)) * np.abs(k).sum(axis=1).max()
        assert (k >= box[0] * 2.0 ** (by - 127)).all() and (k <= box[1] * 2.0 ** (by - 127)).all()
        assert (q @ k.T).max() <= S.scores(q, box[None], np.array([by]))[0] + slack.max()


# ------------------------------------------------------------------------------------------------ allocator

class Model(AllocModel):
    """The allocator's model with compaction: replacements first, in batch order, then the releases."""

    def compact(self, seqs, base, new):
        if len(set(seqs)) < len(seqs):
            raise AllocError("invalid", "repeated")
        for s, b, n in zip(seqs, base, new):
            self._need(s)
            if not 0 <= b <= n <= self.ntok[s]:
                raise AllocError("invalid", "bounds")
        ref, todo = list(self.ref), []
        for i, (s, b, n) in enumerate(zip(seqs, base, new)):
            for blk in sorted({t // self.B for t in range(b, n)}):
                old = self.tables[s][blk]
                if ref[old] > 1:
                    ref[old] -= 1
                    todo.append((i, s, blk, old))
        if len(todo) > len(self.free):
            raise AllocError("oom", "blocks")
        cow, upd = [], []
        for i, s, blk, old in todo:
            new_blk = self.free.pop()
            self.ref[new_blk], self.ref[old] = 1, self.ref[old] - 1
            self.tables[s][blk] = new_blk
            cow.append([old, new_blk])
            upd.append([i, blk, new_blk])
        for s, n in zip(seqs, new):
            left = -(-n // self.B)
            for old in self.tables[s][left:]:
                self.ref[old] -= 1
                if self.ref[old] == 0:
                    self.free.append(old)
            self.tables[s], self.ntok[s] = self.tables[s][:left], n
        return cow, upd


def same(m, a):
    assert list(a.free_list()) == m.free_list_top_first()
    assert [a.refcount(b) for b in range(m.NB)] == m.ref
    for s in m.tables:
        assert list(a.block_table(s)) == m.tables[s] and a.seq_len(s) == m.ntok[s]


@pytest.mark.parametrize("seed", range(12))
def test_random_operations_match_the_model(seed):
    r = np.random.default_rng(seed)
    NB, B = int(r.integers(8, 60)), int(r.choice([1, 2, 4, 8]))
    order = r.permutation(NB)
    m, a = Model(NB, B, order), pa.BlockAllocator(NB, B, order)
    live, nxt, refused = [], 0, 0
    for _ in range(400):
        op = int(r.integers(0, 6))
        if op == 0 or not live:
            m.add_seq(nxt)
            a.add_seq(nxt)
            live.append(nxt)
            nxt += 1
        elif op == 1:
            s, n = int(r.choice(live)), int(r.integers(0, 4 * B))
            try:
                want = m.append_slots(s, n)
            except AllocError:
                with pytest.raises(pa.PAError):
                    a.append_slots(s, n)
            else:
                got = a.append_slots(s, n)
                assert list(got[0]) == want[0] and [tuple(p) for p in got[1]] == want[1]
        elif op == 2 and len(live) < 8:
            s = int(r.choice(live))
            m.fork(s, nxt)
            a.fork(s, nxt)
            live.append(nxt)
            nxt += 1
        elif op == 3:
            s = live.pop(int(r.integers(0, len(live))))
            m.free_seq(s)
            a.free_seq(s)
        else:
            seqs = [int(x) for x in r.permutation(live)[: int(r.integers(1, len(live) + 1))]]
            new = [int(r.integers(0, m.ntok[s] + 1)) for s in seqs]
            base = [int(r.integers(0, n + 1)) for n in new]
            if r.random() < 0.1:
                new[0] = m.ntok[seqs[0]] + 1
            if r.random() < 0.1 and len(seqs) > 1:
                seqs[0] = seqs[1]
            try:
                want = m.compact(seqs, base, new)
            except AllocError as e:
                refused += 1
                with pytest.raises(pa.PAError) as x:
                    a.compact_batch(seqs, base, new, table_updates=True)
                assert x.value.status == (pa.PA_ERR_OOM if e.kind == "oom" else INV)
            else:
                if r.random() < 0.5:
                    cow, upd = a.compact_batch(seqs, base, new, table_updates=True)
                    assert upd.tolist() == want[1]
                else:
                    cow = a.compact_batch(seqs, base, new)
                assert cow.tolist() == want[0]
        same(m, a)
    assert seed or refused > 0
    b = pa.BlockAllocator.from_state(a.export_state())
    same(m, b)


def test_replacements_are_never_blocks_that_the_batch_releases():
    """Sequence 0 gives its tail back in the same call in which sequence 1 needs a block: the tail's tokens are still to
    be moved, so the call is refused rather than served from it."""
    a = pa.BlockAllocator(6, 4)
    a.add_seq(0)
    a.append_slots(0, 16)
    a.add_seq(1)
    a.append_slots(1, 8)
    a.fork(1, 2)
    before = a.export_state()
    with pytest.raises(pa.PAError) as e:
        a.compact_batch([0, 1], [0, 0], [4, 4])
    assert e.value.status == pa.PA_ERR_OOM and np.array_equal(a.export_state(), before)
    assert a.compact_batch([0], [0], [4]).size == 0
    cow = a.compact_batch([1], [0], [4])
    assert cow.tolist() == [[4, 3]]              # the block released last is handed out first


def test_compact_batch_refuses():
    a = pa.BlockAllocator(8, 4)
    for s in (0, 1):
        a.add_seq(s)
        a.append_slots(s, 6)
    a.fork(0, 2)
    before = a.export_state()
    for args in [([5], [0], [1]), ([0, 0], [0, 0], [1, 1]), ([0], [-1], [1]), ([0], [2], [1]), ([0], [0], [7])]:
        with pytest.raises(pa.PAError) as e:
            a.compact_batch(*args)
        assert e.value.status == INV
    with pytest.raises(pa.PAError):
        a.compact_batch([0, 1], [0], [1, 1])
    L, i32 = pa.load(), lambda *x: (ctypes.c_int32 * len(x))(*x)  # noqa: E731
    n = ctypes.c_int(9)
    pairs, upd = (ctypes.c_int64 * 8)(), i32(*range(12))
    call = lambda *x: L.pa_alloc_compact_batch(a._h, 1, i32(0), i32(0), i32(6), *x)  # noqa: E731
    assert call(pairs, 1, ctypes.byref(n), None, 0, None) == INV          # two shared blocks, room for one pair
    assert call(None, 8, ctypes.byref(n), None, 0, None) == INV
    assert call(pairs, 8, ctypes.byref(n), upd, 1, ctypes.byref(n)) == INV
    assert L.pa_alloc_compact_batch(None, 0, None, None, None, None, 0, None, None, 0, None) == INV
    assert L.pa_alloc_compact_batch(a._h, 1, None, None, None, None, 0, None, None, 0, None) == INV
    assert L.pa_alloc_compact_batch(a._h, -1, None, None, None, None, 0, None, None, 0, None) == INV
    assert np.array_equal(a.export_state(), before)
    assert L.pa_alloc_compact_batch(a._h, 0, None, None, None, None, 0, None, None, 0, None) == OK
    assert call(pairs, 2, ctypes.byref(n), upd, 2, None) == OK and n.value == 2
