"""64-bit forms of the quantised cache and of attention over it, for the tests (not collected by pytest).

Everything here is numpy in float64, from the definitions: e4m3 values by rounding to the grid, attention as two
sums.  `attend` also returns how far a kernel that follows the arithmetic below may be from it, element by element.
"""
from __future__ import annotations

import math

import numpy as np
import torch

TORCH_DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E_MIN, E_MAX = -40, 40


def e4m3_decode(bits: np.ndarray) -> np.ndarray:
    """float64 values of e4m3 bit patterns (0x7f and 0xff are NaN)."""
    b = bits.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e.astype(np.float64) - 10))
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b & 0x80, -v, v)


_GRID = e4m3_decode(np.arange(0x7F, dtype=np.uint8))      # the finite non-negative values, ascending


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 bit patterns of float64 values: ties to the even pattern, saturating, NaN to 0x7f."""
    a = np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)).clip(max=448.0)
    hi = np.searchsorted(_GRID, a).clip(0, len(_GRID) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    i = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), 0x7F, i | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def quantise(x: np.ndarray):
    """(bit patterns, scale bytes) of float64 rows [..., D]."""
    a = np.nanmax(np.where(np.isnan(x), 0.0, np.abs(x)), axis=-1)
    e = np.full(a.shape, E_MIN)
    for k in range(E_MIN, E_MAX):
        e = np.where(a > 448.0 * 2.0 ** k, k + 1, e)
    return e4m3_encode(x / np.exp2(e.astype(np.float64))[..., None]), (e + 127).astype(np.uint8)


def values(qbits: np.ndarray, sbytes: np.ndarray) -> np.ndarray:
    e = np.clip(sbytes.astype(np.int64) - 127, E_MIN, E_MAX).astype(np.float64)
    return e4m3_decode(qbits) * np.exp2(e)[..., None]


def attend(q, k, v, ev, see, scale, split_p, p_fp16):
    """Attention rows and their error bound.  q [R, D], k, v [L, D] float64; ev [L] the exponents of V's scales (zeros
    for a 16-bit cache); see [R, L] bool.  Returns out [R, D] and tol [R, D] for an fp32 result.

    The kernels compute s_t = scale (q . k_t) log2 e in fp32, y_t = s_t + ev_t, p_t = 2^(y_t - M), M a running maximum
    of y, acc = sum p_t V_t / 2^ev_t with p rounded, l = sum p_t 2^-ev_t, out = acc / l.
      * s: D products summed in fp32, in D / 16 or fewer steps of at most 2^-22 (a tensor core may truncate) of
        A_t = scale sum |q_d k_td| log2 e each: D / 16 * 2^-22 A_t; four more roundings of |s| and |y|: 2^-24 each;
        as a relative error of p: times ln 2.  2^x by the hardware: 2^-22.
      * these act on numerator and denominator alike: twice.
      * p rounded to fp16: 2^-11, or as a high and a low part 2^-21; to two bf16 parts: 2^-16; in fp16 parts, below
        2^-14 of the reference, an absolute 2^-25 per key instead.
      * sums of up to L terms in fp32, in steps: L / 16 of 2^-22, no more than 64 steps counting (errors of the
        running sum are relative to it, and partial sums of at most 1024 keys join pairwise).
    """
    s = scale * math.log2(math.e) * (q @ k.T)
    A = scale * math.log2(math.e) * (np.abs(q) @ np.abs(k).T)
    s = np.where(see, s, -np.inf)
    y = s + ev[None]
    top = s.max(axis=1, keepdims=True, initial=-np.inf)
    top = np.where(np.isfinite(top), top, 0.0)
    w = np.exp2(s - top)
    l = w.sum(axis=1, keepdims=True)
    empty = l == 0
    l = np.where(empty, 1.0, l)
    vv = np.where(see.any(axis=0)[:, None], v, 0.0)
    out = (w @ vv) / l
    mag = (w @ np.abs(vv)) / l
    D, L = q.shape[1], max(1, k.shape[0])
    seen_max = lambda x: np.where(see, x, 0.0).max(axis=1, keepdims=True, initial=0.0)  # noqa: E731
    d_exp = math.log(2) * (D / 16 * 2.0 ** -22 * seen_max(A) + 4 * 2.0 ** -24 * seen_max(np.abs(y) + np.abs(s))) + 2.0 ** -22
    d_p = 2.0 ** -11 if not split_p else (2.0 ** -21 if p_fp16 else 2.0 ** -16)
    d_sum = 2 * min(64, L / 16 + 1) * 2.0 ** -22
    tol = (2 * d_exp + d_p + d_sum) * mag
    if p_fp16:
        M = np.where(see, y, -np.inf).max(axis=1, keepdims=True, initial=-np.inf)
        M = np.where(np.isfinite(M), M, 0.0)
        tiny = 2.0 ** -25 * (see @ (np.abs(vv) / np.exp2(ev)[:, None])) * np.exp2(M - top) / l
        tol = tol + tiny
    return np.where(empty, 0.0, out), np.where(empty, 0.0, tol)


def close(got: torch.Tensor, want: np.ndarray, tol: np.ndarray, what: str):
    """Every element of got within tol of want, plus the rounding to its own type."""
    g = got.double().cpu().numpy()
    lim = tol + HALF_STEP[got.dtype] * (np.abs(want) + tol) + 2.0 ** -25 * (got.dtype == torch.float16) + 1e-30
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    bad = np.abs(g - want) > lim
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} elements off, worst "
                           f"{float((np.abs(g - want) / lim).max()):.2f} times the bound")


def to64(t: torch.Tensor) -> np.ndarray:
    return t.double().cpu().numpy()


def rows_like_a_model(gen: torch.Generator, shape, dtype) -> torch.Tensor:
    """K or V rows [..., H, D]: channels of different size, tokens of very different norm."""
    x = torch.randn(shape, generator=gen)
    ch = torch.exp(0.5 * torch.randn(shape[-2:], generator=gen))
    tok = torch.exp(1.0 * torch.randn(shape[:-1], generator=gen))[..., None]
    return (0.5 * x * ch * tok).to(dtype)
