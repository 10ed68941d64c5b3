"""Plain implementations of what stands around the halves of a decode step, and
what its GPU tests allow.

* norm, codes: the header defines every operation but the mean as one fp32
  rounding, and the mean goes into fp32 only once, from a sum good to 2^-40, so
  ``norm`` restates them in float32 numpy and results are compared bit by bit.
* 8-bit linear layer: the sum is a whole number, what follows is one fp32 rounding
  per operation, a 16-bit result one more; ``linear8`` restates them and results
  are compared bit by bit.
* continuations: totals in float64. A sum of exponentials is off by at most 2^-22
  of itself: each term by 2^-23 from the argument below one (a float up to 32 in
  size that is rounded twice is off by 2^-19, but only for terms of 2^-16 and less
  of the largest), 2^-22 from the exponential instruction; sums of 32 terms and of
  256 threads add 40 roundings of 2^-24 at random signs and at most 40 * 2^-24. So
  log of it is off by at most 2^-21 + 2^-18.6 and a total by that and its own
  rounding: LSE_OFF. Parents and tokens are equal wherever totals differ by more
  than twice that; tests draw logits that do.
* reordering: bytes move, so results are equal.
"""

from __future__ import annotations

import numpy as np
import torch

LSE_OFF = 2.0 ** -21 + 40 * 2.0 ** -24
NUMPY = {"f32": np.float32, "f16": np.float16}
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def f32(t) -> np.ndarray:
    return t.float().cpu().numpy()


def rounded(a: np.ndarray, dtype: str) -> torch.Tensor:
    """A float32 array rounded once to dtype."""
    return torch.from_numpy(np.ascontiguousarray(a)).to(TORCH[dtype])


def codes(y: np.ndarray):
    """(codes int8, scales float32) of rows y float32."""
    f = np.float32
    top = np.abs(y).max(-1)
    with np.errstate(all="ignore"):
        scale = np.where(np.isfinite(top), (top / f(127)).astype(f), f("nan"))
        q = np.clip(np.rint((y / scale[:, None]).astype(f)), -127, 127)
    q = np.where(scale[:, None] > 0, q, 0)
    return q.astype(np.int8), scale.astype(f)


def norm(x: np.ndarray, residual, weight, eps: float):
    """(t, y) float32 of rows x float32."""
    f = np.float32
    with np.errstate(all="ignore"):
        t = x if residual is None else (x + residual).astype(f)
        mean = np.square(t.astype(np.float64)).sum(-1) / x.shape[-1]
        y = (t * (1.0 / np.sqrt(mean + eps)).astype(f)[:, None]).astype(f)
        return t, y if weight is None else (y * weight.astype(f)).astype(f)


def linear8(x: torch.Tensor, x_scales, w: torch.Tensor, scales, bias, residual, dtype: str) -> torch.Tensor:
    """x (B, in) and w (out, in) int8 tensors; the rest float32 numpy arrays or None."""
    f = np.float32
    total = (x.double() @ w.double().T).cpu().numpy()     # whole numbers below 2^53
    with np.errstate(all="ignore"):
        y = total.astype(f) * (scales[None] * x_scales[:, None]).astype(f)
        y = (y + (0 if bias is None else bias[None])).astype(f)
        if residual is not None:
            y = (y + residual).astype(f)
    return rounded(y, dtype)


def select(logits: np.ndarray, scores: np.ndarray, n_out: int, done=None, end_token=0):
    """(scores float64, parents, tokens) of one search: logits (beams, vocab), scores (beams,) in float64."""
    beams, vocab = logits.shape
    total = np.full((beams, vocab), -np.inf)
    for j in range(beams):
        if not np.isfinite(scores[j]):
            continue
        if done is not None and done[j]:
            total[j, end_token] = scores[j]
            continue
        z = logits[j].astype(np.float64)
        if np.isnan(z).any() or np.isposinf(z).any() or np.isneginf(z).all():
            continue
        top = z.max()
        with np.errstate(over="ignore"):
            total[j] = (z - (top + np.log(np.exp(z - top).sum()))) + scores[j]
    flat = total.ravel()
    order = np.argsort(-flat, kind="stable")[:n_out]
    out, parents, tokens = np.full(n_out, -np.inf), np.zeros(n_out, np.int32), np.zeros(n_out, np.int32)
    for i, at in enumerate(order):
        if flat[at] > -np.inf:
            out[i], parents[i], tokens[i] = flat[at], at // vocab, at % vocab
    return out, parents, tokens
