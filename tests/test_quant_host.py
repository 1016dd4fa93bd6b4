"""Refusals of the quantised cache's and the tree attention's calls, without a GPU: placeholder addresses are never
dereferenced, because validation fails first."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _quant_ref as R
import paged_kv_cache_302_gb300 as pa

A = [0x1000 * (i + 1) for i in range(12)]        # aligned placeholder addresses
F16, BF16, F32, E4M3 = pa.PA_F16, pa.PA_BF16, pa.PA_F32, pa.PA_E4M3
INV, UNS, OK = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED, pa.PA_OK


def write(k=A[0], v=A[1], qp=A[2], sc=A[3], slots=A[4], T=1, NB=4, B=16, H=2, D=128, dt=BF16):
    return pa.load().pa_reshape_and_cache_quant(k, v, qp, sc, slots, T, NB, B, H, D, dt, None, None)


def read(dst=A[0], nd=4, qp=A[1], sc=A[2], ns=4, pairs=A[3], n=1, B=16, H=2, D=128, dt=BF16):
    return pa.load().pa_dequant_blocks(dst, nd, qp, sc, ns, pairs, n, B, H, D, dt, None, None)


def decode(out=A[0], odt=F32, q=A[1], qdt=BF16, qp=A[2], sc=A[3], tab=A[4], ctx=A[5], N=1, Hq=8, H=2, D=128, B=16,
           MB=4, NB=4, mc=64, pt=0, ws=A[6], wsb=1 << 30):
    return pa.load().pa_decode_quant(out, odt, q, qdt, qp, sc, tab, ctx, N, Hq, H, D, B, MB, NB, mc, 0.1, pt, ws, wsb,
                                     None, None, None)


def tree(out=A[0], odt=F32, q=A[1], qdt=BF16, pool=A[2], sc=None, kdt=BF16, tab=A[3], ctx=A[4], qs=A[5], mask=A[6],
         W=1, N=1, T=4, Hq=8, H=2, D=128, B=16, MB=4, NB=4, mq=4, ws=A[7], wsb=1 << 30):
    return pa.load().pa_decode_tree(out, odt, q, qdt, pool, sc, kdt, tab, ctx, qs, mask, W, N, T, Hq, H, D, B, MB, NB,
                                    mq, 0.1, ws, wsb, None, None)


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kw, status", [
    (dict(dt=F32), UNS), (dict(dt=E4M3), UNS), (dict(D=96), UNS), (dict(D=256), UNS), (dict(B=4), UNS),
    (dict(B=64), UNS), (dict(H=0), INV), (dict(qp=None), INV), (dict(sc=None), INV), (dict(qp=A[2] + 8), INV),
    (dict(sc=A[2] + 4), INV)])
def test_cache_calls_refuse(call, kw, status):
    assert call(**kw) == status and pa.last_error()


def test_write_and_read_refuse_their_own():
    assert write(T=-1) == INV and write(k=A[0] + 2) == INV and write(slots=None) == INV
    assert write(NB=1 << 27, B=16) == UNS and "2^31" in pa.last_error()
    assert read(n=-1) == INV and read(pairs=None) == INV and read(nd=0) == INV and read(dst=A[0] + 2) == INV
    # nothing to do is no error, whatever the pointers
    assert write(T=0, k=None, v=None) == OK and read(n=0, dst=None) == OK


@pytest.mark.parametrize("kw, status", [
    (dict(qdt=F32), UNS), (dict(qdt=E4M3), UNS), (dict(odt=F16), UNS), (dict(Hq=18), UNS), (dict(Hq=7), INV),
    (dict(D=96), UNS), (dict(B=4), UNS), (dict(N=0), INV), (dict(MB=0), INV), (dict(mc=0), INV), (dict(pt=48), INV),
    (dict(pt=-2), INV), (dict(ws=None), INV), (dict(wsb=16), INV), (dict(q=A[1] + 2), INV), (dict(sc=None), INV),
    (dict(qp=A[2] + 8), INV), (dict(NB=1 << 27), UNS), (dict(tab=None), INV)])
def test_decode_quant_refuses(kw, status):
    assert decode(**kw) == status and pa.last_error()


@pytest.mark.parametrize("kw, status", [
    (dict(qdt=F32), UNS), (dict(kdt=F16), UNS), (dict(kdt=F32), UNS), (dict(odt=F16), UNS), (dict(Hq=7), INV),
    (dict(Hq=258), UNS), (dict(D=32), UNS), (dict(B=4), UNS), (dict(N=0), INV), (dict(N=65536), INV),
    (dict(W=0), INV), (dict(mq=33), INV), (dict(mq=-1), INV), (dict(kdt=E4M3), INV), (dict(sc=A[8]), INV),
    (dict(ws=None), INV), (dict(wsb=16), INV), (dict(out=A[0] + 8), INV), (dict(mask=None), INV), (dict(T=-1), INV),
    (dict(NB=1 << 27), UNS)])
def test_decode_tree_refuses(kw, status):
    assert tree(**kw) == status and pa.last_error()


def test_decode_tree_with_nothing_to_do():
    assert tree(T=0, q=None) == OK and tree(mq=0, out=None) == OK


def test_tree_workspace():
    need = pa.pa_decode_tree_workspace_bytes(16, 32, 8, 128, 63)
    assert need > 0
    for bad in [(0, 32, 8, 128, 8), (1, 31, 8, 128, 8), (1, 32, 8, 96, 8), (1, 32, 8, 128, 0)]:
        with pytest.raises(pa.PAError):
            pa.pa_decode_tree_workspace_bytes(*bad)


def test_block_moves_of_a_quantised_cache_are_counted_in_its_bytes():
    L = pa.load()
    # 2 * 8 tokens * 1 head * 1 scale byte is one 16-byte vector; half of it is not
    assert L.pa_copy_blocks(None, None, 0, 4, 8, 1, 1, E4M3, None, None) == OK
    assert L.pa_copy_blocks(None, None, 0, 4, 4, 1, 1, E4M3, None, None) == UNS
    assert L.pa_copy_blocks(A[0], None, 1, 4, 8, 1, 1, E4M3, None, None) == INV
    assert L.pa_copy_blocks(A[0], A[1], 1, 4, 8, 1, 8, F32, None, None) == UNS
    assert L.pa_swap_blocks(A[0], 4, A[1], 4, None, 0, 4, 1, 1, E4M3, None, None) == UNS
    # the attention and write calls of the 16-bit cache refuse it
    assert L.pa_reshape_and_cache(A[0], A[1], A[2], A[3], 1, 4, 16, 1, 128, E4M3, None, None) == UNS


def test_python_refuses_before_the_library_is_called():
    qp = torch.zeros(4, 2, 2, 16, 64, dtype=torch.float8_e4m3fn)
    sc = torch.zeros(4, 2, 2, 16, dtype=torch.uint8)
    k = torch.zeros(3, 2, 64, dtype=torch.float16)
    slots = torch.zeros(3, dtype=torch.int64)

    def refused(f, *a, **kw):
        with pytest.raises(pa.PAError):
            f(*a, **kw)

    refused(pa.pa_reshape_and_cache_quant, k, k, qp, sc, slots)                      # host tensors
    refused(pa.pa_reshape_and_cache_quant, k, k, qp.half(), sc, slots)               # not 8-bit
    refused(pa.pa_reshape_and_cache_quant, k, k, qp, sc[:3], slots)                  # scales of another cache
    refused(pa.pa_reshape_and_cache_quant, k[:, :1], k, qp, sc, slots)               # other heads
    refused(pa.pa_reshape_and_cache_quant, k, k, qp, sc, slots[:2])
    refused(pa.pa_dequant_blocks, torch.zeros(4, 8, 2, 2, 64, dtype=torch.float16), qp, sc, slots.view(-1, 1))
    refused(pa.pa_dequant_blocks, torch.zeros(4, 16, 2, 2, 64, dtype=torch.float16), qp, sc, slots.view(-1, 1))
    q = torch.zeros(2, 4, 64, dtype=torch.float16)
    tab, ctx = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    refused(pa.pa_decode_quant, q, q[:, :, :32], qp, sc, tab, ctx, 8)
    refused(pa.pa_decode_quant, q, q, qp, sc, tab[:1], ctx, 8)
    mask, qs = torch.zeros(2, 1, dtype=torch.int32), torch.tensor([0, 1, 2], dtype=torch.int32)
    refused(pa.pa_decode_tree, q, q, qp, tab, ctx, qs, mask, 1)                      # e4m3 pool without scales
    refused(pa.pa_decode_tree, q, q, qp, tab, ctx, qs[:2], mask, 1, scales=sc)
    refused(pa.pa_decode_tree, q, q, qp, tab, ctx, qs, mask[:1], 1, scales=sc)
    refused(pa.pa_copy_blocks, qp.view(4, -1), torch.zeros(1, 2, dtype=torch.int64))


def test_reference_format_agrees_with_torch():
    """The tests' own e4m3 tables against torch's conversion, over every pattern and a dense set of values."""
    bits = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(bits).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3_decode(bits), t, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 40001), R._GRID, (R._GRID[1:] + R._GRID[:-1]) / 2])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    exact = x.astype(np.float32) == x
    assert np.array_equal(R.e4m3_encode(x)[exact], want[exact])
    # every row lies within 448 of its scale and above half of that
    q, e = R.quantise(np.random.default_rng(0).standard_normal((200, 64)) * np.exp2(np.arange(200.0) - 100)[:, None])
    assert e.min() == 87 and e.max() == 127 + 40 and (np.abs(R.e4m3_decode(q)) <= 448).all()


@pytest.mark.parametrize("scale", [0.0, -0.125, float("nan"), float("inf")])
def test_tree_refuses_scales_that_are_not_positive_numbers(scale):
    assert pa.load().pa_decode_tree(A[0], F32, A[1], BF16, A[2], None, BF16, A[3], A[4], A[5], A[6], 1, 1, 4, 8, 2, 128, 16,
                                    4, 4, 4, scale, A[7], 1 << 30, None, None) == INV
    assert "scale" in pa.last_error()


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e4m3fn, torch.bfloat16])
@pytest.mark.parametrize("shape", [(4, 8, 1, 16, 64), (4, 2, 8, 16, 64), (4, 8, 16, 2, 64), (4, 8, 3, 16, 64)])
def test_block_moves_refuse_pools_of_another_shape(dtype, shape):
    """The size of a block counts K and V once each: a pool whose third dimension is not 2 would be moved in blocks of
    another size than its own, past its end among other places."""
    pool, pairs = torch.zeros(shape, dtype=torch.uint8).to(dtype), torch.zeros(1, 2, dtype=torch.int64)
    for move in (lambda: pa.pa_copy_blocks(pool, pairs), lambda: pa.pa_swap_blocks(pool, pool, pairs)):
        with pytest.raises(pa.PAError, match="pool is "):
            move()


def test_block_moves_refuse_scales_of_another_shape():
    for shape in ((4, 8, 1, 16), (4, 2, 8, 16), (4, 8, 2)):
        with pytest.raises(pa.PAError, match="pool is "):
            pa.pa_copy_blocks(torch.zeros(shape, dtype=torch.uint8), torch.zeros(1, 2, dtype=torch.int64))


def test_a_workspace_made_by_a_call_belongs_to_the_calls_stream(monkeypatch):
    """Memory let go at the end of a call may serve the stream it was taken under at once: that has to be the stream the
    kernels run on."""
    current, seen = [None], []

    class Under:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current[0] = self.stream

        def __exit__(self, *exc):
            current[0] = None

    class Stream:
        cuda_stream = 0x77

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", Under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: ptr)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (seen.append(current[0]), empty(*a, **kw))[1])
    mine = empty(64, dtype=torch.uint8)
    assert pa._workspace(mine, 64, "cpu", Stream()) is mine and seen == []
    assert pa._workspace(None, 64, "cpu", Stream()).numel() == 64 and seen == [0x77]
    assert pa._workspace(None, 64, "cpu", None).numel() == 64 and seen == [0x77, None]


_NAMED = """
import paged_kv_cache_302_gb300 as pa
L, size = pa.load(), pa.pa_decode_workspace_bytes
for shape in ((1, 32, 8, 128, 1000), (1, 32, 8, 128, 20000), (256, 32, 8, 128, 16384), (8, 56, 8, 128, 32768)):
    assert size(*shape) == size(*shape, 4096), shape
assert size(256, 32, 8, 128, 16384) < pa.PA_STATIC_WORKSPACE_BYTES < size(256, 32, 8, 128, 16384, 512)
st = L.pa_decode_no_alloc(*([0x1000, pa.PA_BF16] + [0x1000] * 4 + [256, 32, 8, 128, 16, 1024, 4096, 16384, 0.1, 0,
                                                                  pa.PA_BF16, None, None, None]))
assert st == pa.PA_ERR_CUDA, pa.last_error()      # past the check of sizes, to the device that is not there
"""


def test_a_named_partition_length_holds_for_the_sizes_of_every_decode():
    """PA_DECODE_PARTITION sets what partition_tokens = 0 stands for: the workspace is that length's, and batches that fit
    the built-in workspace with it are served."""
    env = {**os.environ, "PA_DECODE_PARTITION": "4096", "CUDA_VISIBLE_DEVICES": ""}
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _NAMED], env=env, cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
