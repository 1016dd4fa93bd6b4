"""64-bit forms of key summaries, block selection and compaction, for the tests (not collected by pytest)."""
from __future__ import annotations

import numpy as np
import torch

import _quant_ref as R

E_MIN, E_MAX = -40, 40
BOX_TOP, QUERY_TOP = 127, 511


def least_exponent(a: np.ndarray, top: int) -> np.ndarray:
    """The least e in [E_MIN, E_MAX] with a <= top * 2^e."""
    e = np.full(a.shape, E_MIN)
    for k in range(E_MIN, E_MAX):
        e = np.where(a > top * 2.0 ** k, k + 1, e)
    return e


def box(k: np.ndarray):
    """Summary of the keys k [t, D] float64 of one block: (ints [2, D], scale byte)."""
    some = ~np.isnan(k).all(axis=0)
    lo = np.where(some, np.where(np.isnan(k), np.inf, k).min(axis=0), 0.0)
    hi = np.where(some, np.where(np.isnan(k), -np.inf, k).max(axis=0), 0.0)
    e = int(least_exponent(np.maximum(np.abs(lo), np.abs(hi)).max(), BOX_TOP))
    b = np.stack([np.floor(lo * 2.0 ** -e), np.ceil(hi * 2.0 ** -e)])
    return b.clip(-BOX_TOP, BOX_TOP).astype(np.int8), e + 127


def scores(q: np.ndarray, boxes: np.ndarray, scale_bytes: np.ndarray) -> np.ndarray:
    """Scores [nb] of boxes [nb, 2, D] for the query heads q [G, D] float64 of one KV head."""
    a = np.where(np.isnan(q), 0.0, np.abs(q)).max(axis=1)
    f = least_exponent(a, QUERY_TOP)
    i = np.where(np.isnan(q), 0.0, np.rint(q * np.exp2(-f.astype(np.float64))[:, None])).clip(-QUERY_TOP, QUERY_TOP)
    b = boxes.astype(np.float64)
    s = np.maximum(i[:, None] * b[None, :, 0], i[:, None] * b[None, :, 1]).sum(axis=2)      # [G, nb]
    e = np.clip(scale_bytes.astype(np.int64) - 127, E_MIN, E_MAX).astype(np.float64)
    return (s * np.exp2(f.astype(np.float64))[:, None]).max(axis=0) * np.exp2(e)


def select(score: np.ndarray, top_k: int, sink: int, recent: int) -> np.ndarray:
    """The list [top_k] of one (sequence, KV head)."""
    nb = len(score)
    out = np.full(top_k, -1, dtype=np.int32)
    s = score.copy()
    b = np.arange(nb)
    s[(b < sink) | (b >= nb - recent)] = np.inf
    pick = np.sort(np.lexsort((b, -s))[:top_k])
    out[: len(pick)] = pick
    return out


def keys_of(cache, blocks, h: int, L: int) -> tuple[np.ndarray, np.ndarray, np.ndarray]:
    """K, V [L, D] float64 and the exponents of V's scales [L], of one KV head through a list of physical blocks.
    cache: (pool,) or (qpool bits, scale bytes), on the host."""
    if len(cache) == 1:
        x = cache[0][blocks][:, :, :, h].reshape(-1, 2, cache[0].shape[-1])[:L]
        return x[:, 0], x[:, 1], np.zeros(L)
    q, s = cache[0][blocks][:, h], cache[1][blocks][:, h]             # [nb, 2, B, D], [nb, 2, B]
    x = R.values(q, s).transpose(1, 0, 2, 3).reshape(2, -1, q.shape[-1])[:, :L]
    ev = np.clip(s[:, 1].reshape(-1)[:L].astype(np.int64) - 127, R.E_MIN, R.E_MAX).astype(np.float64)
    return x[0], x[1], ev


def host_cache(c) -> tuple:
    """The cache's tensors as numpy for keys_of: float64 of a 16-bit pool, or bits and bytes."""
    if len(c) == 1:
        return (R.to64(c[0]),)
    return c[0].view(torch.uint8).cpu().numpy(), c[1].cpu().numpy()


def make_cache(g: torch.Generator, NB, H, B, D, dtype, quant):
    """A filled cache on the GPU: (pool,) or (qpool, scales), rows as a model's."""
    x = R.rows_like_a_model(g, (NB, B, 2, H, D), R.TORCH_DT[dtype])
    if not quant:
        return (x.cuda(),)
    q, e = R.quantise(R.to64(x).transpose(0, 3, 2, 1, 4))
    return torch.from_numpy(q).cuda().view(torch.float8_e4m3fn), torch.from_numpy(e).cuda()


def make_tables(g: torch.Generator, ctx, B, MB, NB):
    """Block tables [N, MB] int32 of distinct blocks, entries past each context out of range."""
    t = torch.full((len(ctx), MB), 1 << 30, dtype=torch.int32)
    free = torch.randperm(NB, generator=g).to(torch.int32)
    at = 0
    for s, L in enumerate(ctx):
        n = -(-L // B)
        t[s, :n] = free[at: at + n]
        at += n
    assert at <= NB
    return t


def make_boxes(g: torch.Generator, NB, H, D):
    """Summaries and their scale bytes as a cache's might be, on the host."""
    lo = torch.randint(-127, 100, (NB, H, 1, D), generator=g)
    hi = (lo + torch.randint(0, 60, (NB, H, 1, D), generator=g)).clamp(max=127)
    return torch.cat([lo, hi], 2).to(torch.int8), torch.randint(122, 126, (NB, H), generator=g, dtype=torch.uint8)
