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


@pytest.mark.parametrize("D,G", [(64, 32), (128, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("dtype,big", [("f16", 60000.0), ("bf16", 2.0 ** 18), ("f32", 2.0 ** 18)])
def test_small_elements_of_a_query_count_beside_large_ones(sffn, D, G, dtype, big):
    """One element 10^8 times the others that meets keys of 0: out and lse stay within the fp32 bound of the rest."""
    n, scale = 200, 4.0
    c = Case(sffn, [(n, 1)], 1, D, G, 16, dtype, seed=D + G)
    k, v = c.randn(n, 1, D) * 100, c.randn(n, 1, D)
    k[..., :G] = 0
    q = c.randn(1, 4, D) * 1e-3
    q[..., 3] = big
    sffn.sffn_kv_append(c.cache.handle, c.all, None, k, v)
    out, lse = attend(sffn, c, c.new, q, scale)
    kh, vh = (R.stored(t.float().cpu().numpy(), G) for t in (k, v))
    step, mid, _ = R.group_params(k.float().cpu().numpy(), G)
    ksize = np.repeat(abs(mid.astype(np.float64)) + 15 * step.astype(np.float64), G, axis=-1)
    want, wlse, tol = R.attention(host(q), kh, vh, 1, scale, 0, ksize)
    R.assert_close(host(out), want, tol, dtype, f"attention {dtype}")
    es = 2.0 ** -20 * scale * np.einsum("hd,ld->hl", abs(host(q)[0]), ksize[:, 0]).max(1)
    assert (abs(host(lse)[0] - wlse[0]) <= es + 2.0 ** -20 * np.maximum(1, abs(wlse[0]))).all()
    c.cache.check_error()


# ------------------------------------------------------------------ rows outside a call's sequences

def call_all(sffn, c, batch, heads=4):
    """(queries, keys, values, attention) that append, read-back and attention leave in arrays of sevens."""
    n = batch.n_tokens
    q, k, v = c.randn(n, heads, c.D), c.randn(n, c.hkv, c.D), c.randn(n, c.hkv, c.D)
    qo, ko, vo, out = (torch.full_like(t, 7.0) for t in (q, k, v, q))
    sffn.sffn_kv_append(c.cache.handle, batch, q, k, v, qo)
    errors = [flagged(sffn, c)]
    sffn.sffn_kv_gather(c.cache.handle, batch, ko, vo)
    errors.append(flagged(sffn, c))
    sffn.sffn_attend(c.cache.handle, batch, q, out, None, 0.1, 0, c.cache.workspace(batch, heads))
    return (q, k, v), (qo, ko, vo, out), errors + [flagged(sffn, c)]


def flagged(sffn, c):
    try:
        c.cache.check_error()
    except sffn.SffnError as e:
        assert e.status == sffn.SFFN_ERR_DEVICE
        return True
    return False


def held(sffn, c):
    k, v = (torch.empty(c.total, c.hkv, c.D, device="cuda") for _ in range(2))
    sffn.sffn_kv_gather(c.cache.handle, c.all, k, v)
    c.cache.check_error()
    return k, v


@pytest.mark.parametrize("seqs", [1, 3, 40])
def test_rows_before_the_first_start_and_after_the_last_are_ignored(sffn, seqs):
    lens = [(20 + s % 7, 2) for s in range(seqs)]
    c = Case(sffn, lens, 2, 64, 64, 16, seed=seqs)
    c.fill_cache(sffn)
    before = held(sffn, c)
    b = sffn.KvBatch(c.table, c.kv_len, c.new.q_start + 5, c.fresh + 9)        # rows 0 .. 4 and the last four
    (q, k, v), (qo, ko, vo, out), errors = call_all(sffn, c, b)
    assert errors == [False] * 3
    for t in (qo, ko, vo, out):
        assert (t[:5] == 7).all() and (t[5 + c.fresh:] == 7).all()
    rows = slice(5, 5 + c.fresh)
    assert torch.equal(qo[rows], q[rows])
    assert np.array_equal(ko[rows].cpu().numpy(), R.stored(k[rows].cpu().numpy(), 64))
    assert np.array_equal(vo[rows].cpu().numpy(), R.stored(v[rows].cpu().numpy(), 64))
    at = 0
    after = held(sffn, c)
    for n, m in lens:                                                          # nothing before the new positions changed
        for x, y in zip(before, after):
            assert torch.equal(x[at:at + n - m], y[at:at + n - m])
        at += n
    want, _ = attend(sffn, c, c.new, q[rows].contiguous(), 0.1)
    assert torch.equal(out[rows], want)


@pytest.mark.parametrize("seqs", [1, 3, 40])
@pytest.mark.parametrize("what", ["descends early", "descends late", "negative", "past the end"])
def test_starts_out_of_order_write_nothing(sffn, seqs, what):
    lens = [(20 + s % 7, 2) for s in range(seqs)]
    c = Case(sffn, lens, 2, 64, 64, 16, seed=seqs)
    c.fill_cache(sffn)
    before = held(sffn, c)
    good = c.new.q_start.clone()
    if what == "descends early":
        c.new.q_start[0] = good[1] + 1
    elif what == "descends late":
        c.new.q_start[seqs] = good[seqs - 1] - 1          # one sequence: negative too
    elif what == "negative":
        c.new.q_start[0] = -1
    else:
        c.new.q_start[seqs] = c.fresh + 1
    _, outs, errors = call_all(sffn, c, c.new)
    assert errors == [True] * 3
    assert all((t == 7).all() for t in outs)
    assert all(torch.equal(x, y) for x, y in zip(before, held(sffn, c)))
    c.new.q_start.copy_(good)
    _, _, errors = call_all(sffn, c, c.new)
    assert errors == [False] * 3


@pytest.mark.parametrize("seqs", [31, 32, 33, 129, 700])
def test_places_of_few_and_many_sequences(sffn, seqs):
    """Up to 32 sequences are looked at by each warp, more by the block together: none to five rows each, some without a place."""
    lens = [((7 * s) % 23, (5 * s) % 6) for s in range(seqs)]
    c = Case(sffn, lens, 1, 64, 32, 16, seed=seqs)
    k, v = c.randn(c.fresh, 1, 64), c.randn(c.fresh, 1, 64)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    sffn.sffn_kv_append(c.cache.handle, c.new, None, k, v)
    sffn.sffn_kv_gather(c.cache.handle, c.new, ko, vo)
    placed = np.concatenate([np.arange(n - m, n) >= 0 for n, m in lens])
    for got, rows in ((ko, k), (vo, v)):
        want = R.stored(rows.cpu().numpy(), 32)
        want[~placed] = 0
        assert np.array_equal(got.cpu().numpy(), want)
    c.cache.check_error()


# ------------------------------------------------------------------ pages outside a window

@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (128, 64), (256, 16)])
@pytest.mark.parametrize("window", [1, 17, 40, 100])
def test_pages_before_the_window_may_be_gone(sffn, D, P, window):
    """Page ids no row of the call sees are replaced by invalid ones: the same bits and no error. A page that is seen in
    part is still looked at."""
    lens = [(300, 1), (250, 9), (64, 64), (33, 2), (129, 3)]
    c = Case(sffn, lens, 2, D, 64, P, seed=window + P)
    c.fill_cache(sffn)
    q = c.randn(c.fresh, 16, D)
    want, wlse = attend(sffn, c, c.new, q, 0.1, window)
    c.cache.check_error()
    first = [max(0, n - m - window + 1) // P for n, m in lens]                # first page that is seen
    gone = c.table.clone()
    for s, f in enumerate(first):
        gone[s, :f] = -1 if s % 2 else c.n_pages + 5
        gone[s, -(-lens[s][0] // P):] = -7
    assert sum(first) > 0
    b = sffn.KvBatch(gone, c.kv_len, c.new.q_start, c.fresh)
    out, lse = attend(sffn, c, b, q, 0.1, window)
    c.cache.check_error()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    gone[0, first[0]] = -1
    attend(sffn, c, b, q, 0.1, window)
    assert flagged(sffn, c)


# ------------------------------------------------------------------ what stands at positions

@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("j", [35, 63, 100, 126, 129])
def test_a_visible_nan_value_is_seen_whatever_its_weight(sffn, dtype, window, j):
    """Scores so far apart that most weights are 0: the NaN channels of a position are NaN in every row that sees it, in
    units that all rows see whole and in the others, and in no other row or channel."""
    lens = [(131, 3)]
    c = Case(sffn, lens, 1, 128, 64, 16, dtype, seed=j)
    k, v = c.fill_cache(sffn)
    v = v.clone()
    v[j, 0, 70] = float("nan")                           # channels 64 .. 127
    sffn.sffn_kv_append(c.cache.handle, c.all, None, k, v)
    q = c.randn(3, 16, 128)
    out, lse = attend(sffn, c, c.new, q, 60.0, window)
    sees = torch.tensor([j <= p and (not window or j > p - window) for p in (128, 129, 130)], device="cuda")
    assert torch.equal(out[..., 64:].isnan(), sees[:, None, None].expand(3, 16, 64))
    assert out[..., :64].isfinite().all() and lse.isfinite().all()
    c.cache.check_error()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("D,G", [(64, 64), (128, 32), (256, 128)])
def test_huge_values_a_row_does_not_see_leave_its_bits_alone(sffn, D, G, dtype):
    """The last of three tokens and the positions before the first one's window get values of 60000 (the second's window
    begins within the change): every row that does not see them has the bits it had."""
    lens, window = [(150, 3)], 70
    c = Case(sffn, lens, 1, D, G, 16, dtype, seed=D)
    k, v = c.fill_cache(sffn)
    q = c.randn(3, 4, D)
    want, wlse = attend(sffn, c, c.new, q, 1 / math.sqrt(D), window)
    for low, high, same in ((149, 150, [0, 1]), (0, 79, [1, 2]), (0, 78, [0, 1, 2])):
        w = v.clone()
        w[low:high] = 60000.0 * torch.sign(w[low:high])
        sffn.sffn_kv_append(c.cache.handle, c.all, None, k, w)
        out, lse = attend(sffn, c, c.new, q, 1 / math.sqrt(D), window)
        assert torch.equal(out[same], want[same]) and torch.equal(lse, wlse)
        assert torch.equal(out, want) == (len(same) == 3)
    c.cache.check_error()


@pytest.mark.parametrize("D,G", [(64, 32), (128, 64), (128, 128), (256, 64)])
@pytest.mark.parametrize("n", [40, 97, 300])
def test_values_of_very_different_sizes_keep_the_fp32_bound(sffn, D, G, n):
    """Groups from 1e5 down to 1e-3, and one position of 1e5 in all channels whose score is 40 below the others."""
    c = Case(sffn, [(n, 1)], 1, D, G, 32, seed=n)
    k, v = c.randn(n, 1, D), c.randn(n, 1, D)
    v *= torch.logspace(5, -3, D // G, device="cuda").repeat_interleave(G)
    q = c.randn(1, 1, D)
    scale = 1 / math.sqrt(D)
    k[n // 3] = q[0] * (-40 / (scale * q.square().sum()))
    v[n // 3] = 1e5 * torch.sign(v[n // 3])
    sffn.sffn_kv_append(c.cache.handle, c.all, None, k, v)
    out, _ = attend(sffn, c, c.new, q, scale)
    kh, vh = (R.stored(t.cpu().numpy(), G) for t in (k, v))
    step, mid, _ = R.group_params(k.cpu().numpy(), G)
    ksize = np.repeat(abs(mid.astype(np.float64)) + 15 * step.astype(np.float64), G, axis=-1)
    want, _, tol = R.attention(host(q), kh, vh, 1, scale, 0, ksize)
    R.assert_close(host(out), want, tol, "f32", f"attention len {n}")
    c.cache.check_error()


# ------------------------------------------------------------------ limits

@pytest.mark.parametrize("pages", [1, 4, 30, 1000])
@pytest.mark.parametrize("hkv", [1, 4])
def test_the_limit_of_one_call_is_the_documented_one(sffn, pages, hkv):
    """On both sides of the header's bound on rows and table, judged on the host: without a workspace nothing is launched,
    and the message tells which check a call met."""
    import ctypes
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "sffn.h")) as f:
        text = " ".join(f.read().replace("*", " ").split())
    past = int(re.search(r"\(table_stride page_size / 32 \+ (\d+)\) below 2\^31", text)[1])
    c = Case(sffn, [(5, 1)], hkv, 64, 64, 16)
    rows = sffn.RowsC(c.kv_len.data_ptr() // 256 * 256, 4096, 64)              # never read
    heads = 8 * hkv

    def message(n_tokens):
        b = sffn.KvBatchC(c.table.data_ptr(), c.kv_len.data_ptr(), c.new.q_start.data_ptr(), 1, n_tokens, pages)
        rc = sffn._lib.sffn_attend(c.cache.handle, ctypes.byref(b), rows, heads, rows, None, 1.0, 0, 0, None, 0, None)
        assert rc == sffn.SFFN_ERR_INVALID_ARG
        return sffn.last_error()

    each = pages * 16 / 32 + past                                             # units of a tile of eight rows, at most
    most = int((2 ** 31 - 1) / each / hkv) - 1                                 # tokens: heads * n / 8 tiles and one a head
    assert "2^30" in message((2 ** 30) // heads + 1)
    if most * heads <= 2 ** 30:
        assert "too large" in message(most + 1)
        assert "ws is NULL" in message(most - 1)
    else:
        assert "ws is NULL" in message(2 ** 30 // heads)


# ------------------------------------------------------------------ projections

@pytest.mark.parametrize("B", [5, 12, 32])
def test_fp16_rows_of_a_projection_are_taken_as_they_are(sffn, B):
    """Elements from the least subnormal on beside the largest half, which meets codes of 0: nothing of them is lost."""
    n, k, group = 40, 512, 64
    g = gen(B)
    codes = torch.randint(-8, 8, (n, k), generator=g, device="cuda", dtype=torch.int8)
    codes[:, 7] = 0
    scales = 1e4 * (0.5 + torch.rand(n, k // group, generator=g, device="cuda"))
    lin = sffn.Linear.from_weights(codes, scales, max_batch=B)
    x = (torch.randint(-40, 41, (B, k), generator=g, device="cuda") * 2.0 ** -24).half()
    x[:, 7] = 65504.0
    y = torch.empty(B, n, device="cuda", dtype=torch.float16)
    sffn.sffn_linear_forward(lin.handle, x, y, None, lin.workspace(B))
    want, tol = R.linear(host(x), codes.cpu().numpy(), host(scales), None, None, None, group)
    R.assert_close(host(y), want, tol, "f16", f"B {B}")
    lin.check_error()
