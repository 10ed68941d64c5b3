"""The attention half of a decode step on the GPU where its calls can go wrong:
bits of 16-bit rows, rows and pages outside a call's sequences and windows, and
what stands at positions a row does not see."""

import math

import numpy as np
import pytest
import torch

import attn_ref as R
from test_gpu_attention import TORCH, Case, check_linear, gen, host, sffn  # noqa: F401  (sffn is a fixture)

pytestmark = pytest.mark.gpu


def attend(sffn, c, batch, q, scale, window=0):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    sffn.sffn_attend(c.cache.handle, batch, q, out, lse, scale, window, c.cache.workspace(batch, q.shape[1]))
    return out, lse


# ------------------------------------------------------------------ bits of 16-bit rows

@pytest.mark.parametrize("D,G", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_of_16_bit_rows_keeps_fp32_sums(sffn, D, G, dtype):
    """16-bit rows are rounded when they are written and nowhere before: the bound is the one of fp32 rows (keys with 30
    steps, their codes standing for 0 to 30 steps above mid - 15 steps) and half a unit of the result's last place."""
    lens = [(97, 2), (3000, 1), (64, 64)]
    c = Case(sffn, lens, 2, D, G, 16, dtype, seed=D)
    c.fill_cache(sffn)
    q = c.randn(c.fresh, 8, D)
    out, _ = attend(sffn, c, c.new, q, 1 / math.sqrt(D))
    qh, oh, at, row = host(q), host(out), 0, 0
    for n, m in lens:
        want, _, tol = R.attention(qh[row:row + m], c.k[at:at + n], c.v[at:at + n], m, 1 / math.sqrt(D), 0,
                                   c.ksize[at:at + n], None)
        R.assert_close(oh[row:row + m], want, tol, dtype, f"attention len {n} new {m}")
        at, row = at + n, row + m
    c.cache.check_error()
