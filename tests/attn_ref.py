"""Plain implementations of the attention half of a decode step, and the bounds
its GPU tests allow.

``stored`` restates the rounding of cached rows in float32 numpy (one rounding
per operation), so the cache's contents are compared bit by bit. ``attention``
and ``linear`` compute in float64 and return, with the result, the sum of
absolute terms that the bounds are made of:

* linear, fp32 arithmetic: inputs split into two halves carry them to 2^-22;
  the products of a group of at most 128 inputs are summed in at most 8 steps
  of a tensor core, each off by at most 2^-22 of the terms' absolute sum; the
  K/G group sums are added in fp32. Together at most (40 + K/G) 2^-24 of
  sum |w||x|.
* attention: a score is a sum of q * mid and q * step * (2u - 15), or with
  16-bit rows of q * step * 2u and a sum taken off again, so it is off by at most
  2^-20 of scale * sum |q| (|mid| + 15 step), twice the step with 16-bit rows,
  its own rounding included; a weight by that and 2^-20 relative, the
  weighted sum of values by a further 2^-19 of sum p|V|; the normalisation at
  most doubles the first part. With 16-bit rows the product of a weight and a
  step is rounded to a half (2^-11 relative): with step |2u - 15| <= |V| + |mid|
  at most 2^-11 of sum p (|V| + |mid|) more.
* a result rounded to 16 bits is off by a further half unit in the last place.
"""

from __future__ import annotations

import numpy as np

HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def group_params(x: np.ndarray, group: int):
    """(step, mid, u) of rows x (..., D) float32."""
    f = np.float32
    x = x.astype(f)
    g = x.reshape(*x.shape[:-1], -1, group)
    bad = ~np.isfinite(g).all(-1)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        mid = np.clip(lo * f(0.5) + hi * f(0.5), f(-65504), f(65504)).astype(np.float16)
        far = np.maximum(hi - mid.astype(f), mid.astype(f) - lo)
        step = np.minimum(far * (f(1) / f(15)), f(65504)).astype(np.float16)
        mid[bad], step[bad] = np.float16("nan"), 0
        inv = f(1) / (f(2) * step.astype(f))
        u = np.floor((g - mid.astype(f)[..., None]) * inv[..., None] + f(8))
    u = np.where(step[..., None] == 0, f(8), np.clip(u, 0, 15))
    return step, mid, u


def stored(x: np.ndarray, group: int) -> np.ndarray:
    """The values the cache holds for rows x (..., D), float32."""
    step, mid, u = group_params(x, group)
    v = mid.astype(np.float32)[..., None] + step.astype(np.float32)[..., None] * (2 * u.astype(np.float32) - 15)
    return v.reshape(x.shape).astype(np.float32)


def rotate(x: np.ndarray, cs: np.ndarray, style: str) -> np.ndarray:
    """Rows x (n, heads, D) float32 turned by cs (n, R/2, 2), one float32 rounding per operation."""
    x, r = x.astype(np.float32).copy(), cs.shape[1]
    a, b = (slice(0, r), slice(r, 2 * r)) if style == "halves" else (slice(0, 2 * r, 2), slice(1, 2 * r, 2))
    c, s, u, w = cs[:, None, :, 0], cs[:, None, :, 1], x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = u * c - w * s, w * c + u * s
    return x


def attention(q, k, v, n_new: int, scale: float, window: int, ksize=None, vsize=None):
    """One sequence: q (n_new, Hq, D), k, v (len, Hkv, D); ksize
    (len, Hkv, D) |mid| + 15 step of the keys (30 with 16-bit rows); vsize (len, Hkv, D) |V| + |mid|
    if the rows have 16 bits. Returns out, lse and the bound on
    the error of out, all float64."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, hq = k.shape[0], q.shape[1]
    out, lse, tol = np.zeros_like(q), np.full(q.shape[:2], -np.inf), np.zeros_like(q)
    rep = hq // k.shape[1]
    for i in range(n_new):
        p = n - n_new + i
        if p < 0:
            continue
        a = max(0, p - window + 1) if window else 0
        kk, vv = (np.repeat(t[a:p + 1], rep, axis=1) for t in (k, v))
        s = np.einsum("hd,lhd->hl", q[i], kk) * scale
        ks = abs(kk) if ksize is None else np.repeat(ksize[a:p + 1], rep, axis=1)
        es = 2.0 ** -20 * abs(scale) * np.einsum("hd,lhd->hl", abs(q[i]), ks).max(1)
        m = s.max(1)
        w = np.exp(s - m[:, None])
        lse[i] = m + np.log(w.sum(1))
        w /= w.sum(1, keepdims=True)
        out[i] = np.einsum("hl,lhd->hd", w, vv)
        tol[i] = (2 * (es + 2.0 ** -20) + 2.0 ** -19)[:, None] * np.einsum("hl,lhd->hd", w, abs(vv))
        if vsize is not None:
            tol[i] += 2.0 ** -11 * np.einsum("hl,lhd->hd", w, np.repeat(vsize[a:p + 1], rep, axis=1))
    return out, lse, tol


def linear(x, codes, scales, zeros, bias, residual, group: int):
    """float64 result (B, N) and the bound on its error before the final rounding."""
    x = np.asarray(x, dtype=np.float64)
    c = codes.astype(np.float64)
    w = c - (0 if zeros is None else np.repeat(zeros.astype(np.float64), group, axis=1))
    s = np.repeat(scales.astype(np.float64), group, axis=1)
    y = x @ (w * s).T
    # with zeros, the products of codes and of zeros are summed apart
    size = np.abs(x) @ ((np.abs(c) + (0 if zeros is None else np.abs(w - c))) * np.abs(s)).T
    tol = (40 + x.shape[1] / group) * 2.0 ** -24 * size
    if bias is not None:
        y, tol = y + bias, tol + 2.0 ** -23 * np.abs(bias)
    if residual is not None:
        y, tol = y + residual, tol + 2.0 ** -23 * np.abs(residual)
    return y, tol


def assert_close(got, want, tol, dtype: str, what: str) -> None:
    got = np.asarray(got, dtype=np.float64)
    bound = tol + (np.abs(want) + tol) * HALF_ULP[dtype] + (2.0 ** -25 if dtype == "f16" else 0.0)
    off = np.abs(got - want)
    if not off.size:
        return
    worst = np.unravel_index(np.argmax(np.where(bound > 0, off / np.maximum(bound, 1e-300), np.where(off > 0, np.inf, 0))),
                             off.shape)
    assert (off <= bound).all(), f"{what}: off by {off[worst]:.3e}, {bound[worst]:.3e} allowed, at {worst}"
