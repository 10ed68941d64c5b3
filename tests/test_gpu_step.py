"""Norm with 8-bit rows, 8-bit linear layer, continuations and reordering of the
cache against plain implementations (step_ref)."""

import math

import numpy as np
import pytest
import torch

import step_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sffn():
    import __graft_entry__
    __graft_entry__.build()
    from activation_sparse_ffn_gb300 import sffn
    return sffn


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def bits(t):
    return t.contiguous().view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(got, want):
    """Equal bits; any NaN is as good as another."""
    want = want.to(got.device)
    return torch.equal(torch.where(got.isnan(), 0, bits(got)), torch.where(want.isnan(), 0, bits(want))) \
        and torch.equal(got.isnan(), want.isnan())


# ----------------------------------------------------------------- norm

def norm_inputs(rows, width, dtype, seed=0):
    g, t = gen(seed), R.TORCH[dtype]
    x = torch.randn(rows, width, generator=g, device="cuda")
    x[:, :: max(1, width // 3)] *= 10
    return (x.to(t), torch.randn(rows, width, generator=g, device="cuda").to(t),
            1 + 0.2 * torch.randn(width, generator=g, device="cuda"))


def check_norm(sffn, x, r, w, eps, dtype, y_dtype=None):
    rows, width = x.shape
    total, y = torch.empty_like(x), torch.empty(rows, width, dtype=R.TORCH[y_dtype or dtype], device="cuda")
    q, s = torch.empty(rows, width, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    sffn.sffn_norm(x, w, eps, r, total, y, q, s)
    t, want = R.norm(R.f32(x), None if r is None else R.f32(r), None if w is None else R.f32(w), eps)
    codes, scales = R.codes(want)
    assert same(total, R.rounded(t, dtype))
    assert same(y, R.rounded(want, y_dtype or dtype))
    assert same(s, torch.from_numpy(scales))
    assert torch.equal(q.cpu(), torch.from_numpy(codes))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (2, 64), (5, 100), (1, 4099), (2, 8192), (3, 16384), (1, 32768),
                                        (2, 32767), (400, 96), (350, 2056), (310, 8192), (306, 10001)])
def test_norm(sffn, dtype, rows, width):
    x, r, w = norm_inputs(rows, width, dtype)
    check_norm(sffn, x, r, w, 1e-5, dtype)


@pytest.mark.parametrize("dtype,y_dtype", [("bf16", "f32"), ("f32", "f16"), ("f16", "bf16")])
def test_norm_of_another_type(sffn, dtype, y_dtype):
    x, r, w = norm_inputs(5, 1000, dtype)
    check_norm(sffn, x, r, w, 1e-5, dtype, y_dtype)
    check_norm(sffn, x, None, None, 0.0, dtype, y_dtype)


@pytest.mark.parametrize("rows", [6, 400])
@pytest.mark.parametrize("width", [40, 8192])
def test_norm_of_values_at_the_ends_of_the_range(sffn, rows, width):
    x, r, w = norm_inputs(rows, width, "f32", 1)
    x[0] *= 1e30                 # squares past fp32
    x[1] *= 1e-30                # squares below fp32
    x[2] *= 2e-42                # subnormal
    x[3] = 0
    x[4, width // 2] = math.nan
    x[5, 1] = math.inf
    check_norm(sffn, x, None, w, 1e-5, "f32")
    check_norm(sffn, x, None, None, 0.0, "f32")
    x[4, 3] = -math.inf          # beside the NaN
    check_norm(sffn, x, None, w, 0.0, "f32")


def test_norm_places(sffn):
    """Views with longer rows and odd offsets, results in place, what lies beside them untouched."""
    for dtype in ("f32", "bf16"):
        x0, r0, w = norm_inputs(7, 300, dtype, 2)
        t, y = R.norm(R.f32(x0), R.f32(r0), R.f32(w), 1e-6)
        wide = torch.full((7, 333), 7.0, dtype=x0.dtype, device="cuda")
        for off in (0, 1, 8):
            x, r = wide.clone(), wide.clone()
            x[:, off:off + 300], r[:, off:off + 300] = x0, r0
            sffn.sffn_norm(x[:, off:off + 300], w, 1e-6, r[:, off:off + 300], r[:, off:off + 300], x[:, off:off + 300])
            assert same(x[:, off:off + 300], R.rounded(y, dtype)) and same(r[:, off:off + 300], R.rounded(t, dtype))
            for a in (x, r):
                assert bool((a[:, :off] == 7).all()) and bool((a[:, off + 300:] == 7).all())
        odd = torch.empty(7, 301, dtype=torch.int8, device="cuda").fill_(99)
        s = torch.empty(7, device="cuda")
        sffn.sffn_norm(x0, w[:300], 1e-6, r0, codes=odd[:, 1:], scales=s)
        q, _ = R.codes(y)
        assert torch.equal(odd[:, 1:].cpu(), torch.from_numpy(q)) and bool((odd[:, 0] == 99).all())
        heads = x0.view(7, 3, 100)
        out = torch.empty_like(heads)
        sffn.sffn_norm(heads, w, 1e-6, r0, y=out)
        assert same(out.view(7, 300), R.rounded(y, dtype))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 33), (2, 8192), (400, 1024), (2, 65536), (2, 40001)])
def test_quantize(sffn, dtype, rows, width):
    x, _, _ = norm_inputs(rows, width, dtype, 3)
    if rows > 2:
        x[0], x[1, 0], x[2, -1] = 0, math.nan, math.inf
    q, s = torch.empty(rows, width, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    sffn.sffn_quantize(x, q, s)
    codes, scales = R.codes(R.f32(x))
    assert torch.equal(q.cpu(), torch.from_numpy(codes)) and same(s, torch.from_numpy(scales))


def test_quantize_ties_and_small_scales(sffn):
    """Quotients half-way between two codes, scales whose reciprocal is infinite, subnormal rows."""
    half = torch.arange(-126.5, 127, 1.0, device="cuda")
    rows = [torch.cat((half, half.new_tensor([127.0]))) * m for m in (1.0, 2.0 ** -120, 2.0 ** 100, 3e-41, 0.1)]
    x = torch.stack(rows)
    q, s = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(rows), device="cuda")
    sffn.sffn_quantize(x, q, s)
    codes, scales = R.codes(R.f32(x))
    assert torch.equal(q.cpu(), torch.from_numpy(codes)) and same(s, torch.from_numpy(scales))
    assert torch.equal(q[0, :-1].float(), half.round())          # ties go to even


def test_norm_of_no_rows(sffn):
    x = torch.empty(0, 64, device="cuda")
    sffn.sffn_norm(x, None, 1e-5, y=x)
    sffn.sffn_quantize(x, torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))


# ----------------------------------------------------------------- 8-bit linear layer

def linear_inputs(n, k, rows, seed=0, extreme=False):
    g = gen(seed)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randint(-128, 128, (rows, k), generator=g, device="cuda", dtype=torch.int8)
    if extreme:                  # the largest sums: every product 2^14, or -127 * 128
        w.fill_(-128), x.fill_(-128)
        w[n // 2:], x[rows // 2:] = 127, 127
    scales = (0.5 + torch.rand(n, generator=g, device="cuda")) / (5000 * math.sqrt(k))
    xs = 0.5 + torch.rand(rows, generator=g, device="cuda")
    return w, scales, x, xs, torch.randn(n, generator=g, device="cuda"), g


SIZES = [(1, 16, 1), (5, 48, 3), (130, 64, 33), (100, 4096, 7), (129, 1040, 32), (300, 8192, 64), (40, 65536, 9),
         (1000, 2048, 200), (4099, 512, 193), (2433, 11008, 17), (64, 16384, 1), (10240, 1024, 1), (257, 192, 1000),
         (700, 65536, 70), (20000, 64, 40), (128, 1088, 385), (64, 16, 40)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,k,rows", SIZES)
def test_linear8(sffn, dtype, n, k, rows):
    w, scales, x, xs, bias, g = linear_inputs(n, k, rows)
    r = torch.randn(rows, n, generator=g, device="cuda").to(R.TORCH[dtype])
    for with_bias, with_residual in ((True, True), (False, False)):
        L = sffn.Linear8.from_weights(w, scales, bias if with_bias else None, max_batch=rows)
        y = torch.full((rows + 1, n), 7.0, dtype=R.TORCH[dtype], device="cuda")
        sffn.sffn_linear8_forward(L.handle, x, xs, y[:rows], r if with_residual else None, L.workspace(rows))
        L.check_error()
        want = R.linear8(x, R.f32(xs), w, R.f32(scales), R.f32(bias) if with_bias else None,
                         R.f32(r) if with_residual else None, dtype)
        assert same(y[:rows], want)
        assert bool((y[rows] == 7).all())


@pytest.mark.parametrize("n,k,rows", [(40, 65536, 4), (130, 65536, 100), (300, 4096, 300), (33, 1040, 20)])
def test_linear8_largest_sums(sffn, n, k, rows):
    w, scales, x, xs, bias, _ = linear_inputs(n, k, rows, 1, extreme=True)
    L = sffn.Linear8.from_weights(w, scales, bias, max_batch=rows)
    y = torch.empty(rows, n, device="cuda")
    sffn.sffn_linear8_forward(L.handle, x, xs, y, None, L.workspace(rows))
    assert same(y, R.linear8(x, R.f32(xs), w, R.f32(scales), R.f32(bias), None, "f32"))


def test_linear8_of_any_batch_gives_a_token_the_same_bits(sffn):
    w, scales, x, xs, bias, _ = linear_inputs(1500, 3104, 600, 2)
    L = sffn.Linear8.from_weights(w, scales, bias, max_batch=600)
    ws = L.workspace(600)                                       # of the largest batch, for every other
    full = torch.empty(600, 1500, device="cuda")
    sffn.sffn_linear8_forward(L.handle, x, xs, full, None, ws)
    for B in (1, 2, 8, 9, 16, 17, 32, 33, 48, 64, 65, 100, 128, 129, 192, 193, 256, 257, 400):
        y = torch.empty(B, 1500, device="cuda")
        sffn.sffn_linear8_forward(L.handle, x[:B], xs[:B], y, None, ws)
        assert same(y, full[:B]), B


@pytest.mark.parametrize("rows", [1, 9, 40, 150])
def test_linear8_places(sffn, rows):
    """Rows within longer ones, an odd place for y, the residual in y's own place, a token with scale NaN."""
    n, k = 201, 320
    w, scales, x, xs, bias, g = linear_inputs(n, k, rows, 3)
    wide = torch.zeros(rows, k + 48, dtype=torch.int8, device="cuda")
    wide[:, 16:16 + k] = x
    xs[rows // 2] = math.nan
    L = sffn.Linear8.from_weights(w, scales, bias, max_batch=rows)
    y = torch.randn(rows, n + 10, generator=g, device="cuda").bfloat16()
    before = y.clone()
    sffn.sffn_linear8_forward(L.handle, wide[:, 16:16 + k], xs, y[:, 3:3 + n], y[:, 3:3 + n], L.workspace(rows))
    want = R.linear8(x, R.f32(xs), w, R.f32(scales), R.f32(bias), R.f32(before[:, 3:3 + n]), "bf16")
    assert same(y[:, 3:3 + n], want)
    assert torch.equal(y[:, :3], before[:, :3]) and torch.equal(y[:, 3 + n:], before[:, 3 + n:])
    assert bool(y[rows // 2, 3:3 + n].isnan().all()) and int(y.isnan().sum()) == n


def test_linear8_refusals(sffn):
    w, scales, x, xs, bias, _ = linear_inputs(64, 64, 40)
    L = sffn.Linear8(64, 64, max_batch=40)
    y = torch.empty(40, 64, device="cuda")
    ws = L.workspace(40)
    with pytest.raises(sffn.SffnError, match="holds no weights"):
        sffn.sffn_linear8_forward(L.handle, x, xs, y, None, ws)
    sffn.sffn_linear8_pack(L.handle, w, scales, bias)
    wide = torch.zeros(41, 72, dtype=torch.int8, device="cuda")
    for bad in (lambda: sffn.sffn_linear8_forward(L.handle, wide[:40, :64], xs, y, None, ws),          # stride % 16
                lambda: sffn.sffn_linear8_forward(L.handle, wide.view(-1)[8:8 + 64].view(1, 64), xs[:1], y[:1], None, ws),
                lambda: sffn.sffn_linear8_forward(L.handle, torch.zeros(41, 64, dtype=torch.int8, device="cuda"),
                                                  torch.ones(41, device="cuda"), torch.empty(41, 64, device="cuda"), None, ws)):
        with pytest.raises(sffn.SffnError):
            bad()
    if sffn.sffn_linear8_workspace_bytes(L.handle, 40):
        with pytest.raises(sffn.SffnError, match="ws"):
            sffn.sffn_linear8_forward(L.handle, x, xs, y, None, None)


# ----------------------------------------------------------------- continuations

def check_select(sffn, logits, scores, n_out, done=None, end_token=0, fault=False, off=0.0):
    beams = scores.shape[1]
    batch, vocab = scores.shape[0], logits.shape[1]
    H = sffn.Beams(vocab, beams, n_out, max_batch=batch)
    out = torch.empty(batch, n_out, device="cuda")
    parents, tokens = torch.empty(2, batch, n_out, dtype=torch.int32, device="cuda")
    sffn.sffn_beam_select(H.handle, logits, scores, out, parents, tokens, done, end_token, H.workspace(batch))
    if fault:
        with pytest.raises(sffn.SffnError):
            H.check_error()
    H.check_error()
    z, s = logits.double().cpu().numpy(), scores.double().cpu().numpy()
    d = None if done is None else done.cpu().numpy().astype(bool)
    for b in range(batch):
        want, wp, wt = R.select(z[b * beams:(b + 1) * beams], s[b], n_out, None if d is None else d[b], end_token)
        np.testing.assert_array_equal(parents[b].cpu().numpy(), wp)
        np.testing.assert_array_equal(tokens[b].cpu().numpy(), wt)
        got = out[b].double().cpu().numpy()
        live = np.isfinite(want)
        np.testing.assert_array_equal(np.isneginf(got), ~live)
        limit = R.LSE_OFF + 2.0 ** -24 * np.abs(want[live]) + off
        assert (np.abs(got[live] - want[live]) <= limit).all()


def logits_of(rows, vocab, dtype, seed=0):
    return (2.5 * torch.randn(rows, vocab, generator=gen(seed), device="cuda")).to(R.TORCH[dtype])


def scores_of(batch, beams, seed=0):
    return -3 - 4 * torch.rand(batch, beams, generator=gen(1000 + seed), device="cuda")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch,beams,vocab,n_out", [(1, 1, 1, 1), (2, 3, 5, 4), (1, 4, 32000, 8), (3, 5, 50257, 10),
                                                     (2, 8, 2048, 16), (1, 64, 4097, 64), (5, 2, 300, 64), (40, 4, 8193, 4),
                                                     (1, 1, 262145, 50), (16, 16, 33333, 32)])
def test_select(sffn, dtype, batch, beams, vocab, n_out):
    check_select(sffn, logits_of(batch * beams, vocab, dtype), scores_of(batch, beams), n_out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_with_masked_tokens(sffn, dtype):
    z = logits_of(12, 9000, dtype, 1)
    for i, share in enumerate((0.5, 0.99, 0.9995)):
        z[4 * i:4 * i + 4][torch.rand(4, 9000, generator=gen(i), device="cuda") < share] = -math.inf
    z[5] = -math.inf                                            # nothing left
    z[9, :] = -math.inf
    z[9, 8999] = 1.0                                            # one left
    check_select(sffn, z, scores_of(3, 4), 16)
    z[8:12] = -math.inf                                         # a search with nothing left at all
    check_select(sffn, z, scores_of(3, 4), 16)
    # masks of the type's lowest value: such tokens are candidates, after every other
    z = logits_of(4, 700, dtype, 2)
    low = torch.finfo(z.dtype).min
    z[:, 5:] = low
    z[1] = low
    check_select(sffn, z, scores_of(1, 4), 8)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_select_among_equals(sffn, dtype):
    """Ties go to the lowest index: few different logits, the same logits everywhere, beams that are copies."""
    t = R.TORCH[dtype]
    z = torch.randint(0, 3, (6, 20000), generator=gen(0), device="cuda").to(t)
    check_select(sffn, z, torch.tensor([[-1.0, -1.0, -2.0], [-1.0, -4.0, -1.5]], device="cuda"), 20)
    check_select(sffn, torch.full((4, 10000), 0.25, dtype=t, device="cuda"), torch.full((2, 2), -1.0, device="cuda"), 33)
    one = logits_of(1, 5000, dtype, 3)
    check_select(sffn, one.expand(4, -1).contiguous(), torch.full((1, 4), -2.5, device="cuda"), 16)
    z = torch.zeros(2, 300, dtype=t, device="cuda")
    z[:, ::2] = -0.0                                            # zeros of both signs are equal
    check_select(sffn, z, torch.zeros(1, 2, device="cuda"), 5)


def test_select_first_step_and_ended_sequences(sffn):
    z = logits_of(12, 7000, "f32", 4)
    scores = torch.full((3, 4), -math.inf, device="cuda")
    scores[:, 0] = 0
    z[2] = math.nan                                             # of a sequence that is not alive: not looked at
    check_select(sffn, z, scores, 8)
    scores = scores_of(3, 4, 5)
    done = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    done[0, 2] = done[1, :] = True
    z[4] = math.nan                                             # of one that has ended
    check_select(sffn, z, scores, 8, done, end_token=6999)
    check_select(sffn, z, scores, 8, done.to(torch.uint8) * 3, end_token=0)
    scores[1, 1] = -math.inf
    check_select(sffn, z, scores, 8, done, end_token=17)


def test_select_reports_what_has_no_distribution(sffn):
    z, scores = logits_of(8, 3000, "f32", 6), scores_of(2, 4, 6)
    for at, v in (((1, 2999), math.nan), ((6, 0), math.inf)):
        bad = z.clone()
        bad[at] = v
        check_select(sffn, bad, scores, 8, fault=True)
    bad = scores.clone()
    bad[0, 3] = math.nan
    check_select(sffn, z, bad, 8, fault=True)
    bad[0, 3] = math.inf
    check_select(sffn, z, bad, 8, fault=True)


@pytest.mark.parametrize("batch,beams,vocab,n_out,dtype", [(40, 16, 60000, 32, "f32"), (77, 8, 70001, 64, "bf16"),
                                                           (1, 16, 250001, 32, "f16"), (1, 64, 30000, 64, "f32")])
def test_select_of_long_parts(sffn, batch, beams, vocab, n_out, dtype):
    """Rows that a block or two take alone, with more that reaches the first chunk's bound than the list holds; many candidates."""
    check_select(sffn, logits_of(batch * beams, vocab, dtype, 12), scores_of(batch, beams, 12), n_out)


def test_select_of_logits_that_rise_and_fall(sffn):
    """Parts whose largest logits come late, or lie far below those before, and references between -2^22 and 2^22."""
    z = logits_of(6, 60000, "f32", 11)
    at = torch.arange(60000, device="cuda")
    z[0] += at * 0.01
    z[1] -= at * 0.01
    z[2] += (at // 8192) * 90.0
    z[3] -= 4.1e6
    z[4] += 4.1e6
    z[5, :59000] = -1e9
    check_select(sffn, z, scores_of(1, 6, 11), 12, off=2.0 ** -24 * 4.1e6)
    check_select(sffn, z[:1].half(), scores_of(1, 1, 11), 50)


def test_select_of_large_logits(sffn):
    """Logits beyond the range of a whole-number reference, in all chunks or some."""
    z = logits_of(4, 9000, "f32", 7)
    z[0] *= 1e30
    z[1] += 1e7
    z[2, 4000:] -= 3e8
    z[3] *= 3e6
    # a total of size v is rounded to 2^-24 v; sums of fp32 logits this far apart have one term
    check_select(sffn, z, scores_of(1, 4, 7), 12, off=2.0 ** -24 * 1e7)


def test_select_places(sffn):
    """Rows within longer ones at odd places, scores replaced in place, one workspace for every batch."""
    wide = torch.full((24, 6010), math.nan, device="cuda", dtype=torch.bfloat16)
    z = logits_of(24, 6001, "bf16", 8)
    wide[:, 3:6004] = z
    scores = scores_of(6, 4, 8)
    H = sffn.Beams(6001, 4, 4, max_batch=6)
    ws = H.workspace(6)
    for batch in (6, 1, 5, 2):
        out = scores[:batch].clone()
        parents, tokens = torch.empty(2, batch, 4, dtype=torch.int32, device="cuda")
        sffn.sffn_beam_select(H.handle, wide[:4 * batch, 3:6004], out, out, parents, tokens, ws=ws)
        H.check_error()
        for b in range(batch):
            want, wp, wt = R.select(z[4 * b:4 * b + 4].double().cpu().numpy(), scores[b].double().cpu().numpy(), 4)
            np.testing.assert_array_equal(parents[b].cpu().numpy(), wp)
            np.testing.assert_array_equal(tokens[b].cpu().numpy(), wt)
            assert (np.abs(out[b].double().cpu().numpy() - want) <= R.LSE_OFF + 2.0 ** -24 * np.abs(want)).all()


def test_select_workspace_of_a_batch_serves_smaller_ones(sffn):
    for vocab, beams in ((50000, 8), (131072, 4), (1000, 16)):
        H = sffn.Beams(vocab, beams, 16, max_batch=64)
        need = [sffn.sffn_beam_workspace_bytes(H.handle, b) for b in range(1, 65)]
        assert need == sorted(need) and need[0] > 0


# ----------------------------------------------------------------- reordering

def make_caches(sffn, n_layers, n_seq, width, page, hkv, dim, group, seed=0):
    """Caches with the same tables but different n_pages, and a table that names every page once."""
    caches = [sffn.KvCache(n_seq * width + 3 * i, page, hkv, dim, group) for i in range(n_layers)]
    table = torch.randperm(n_seq * width, generator=gen(seed), device="cuda").view(n_seq, width).to(torch.int32)
    return caches, table


def fill(sffn, caches, table, lengths, hkv, dim, seed=0):
    """Random keys and values at every cached position."""
    kv_len = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    start = torch.tensor([0] + np.cumsum(lengths).tolist(), dtype=torch.int32, device="cuda")
    n, g = sum(lengths), gen(seed)
    for c in caches:
        k, v = (torch.randn(n, hkv, dim, generator=g, device="cuda") for _ in range(2))
        if n:
            sffn.sffn_kv_append(c.handle, sffn.KvBatch(table, kv_len, start, n), None, k, v)
    return kv_len


def read(sffn, cache, table, lengths, hkv, dim):
    """[(keys, values)] of every sequence's cached positions."""
    n = sum(lengths)
    if not n:
        return [None] * len(lengths)
    kv_len = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    start = torch.tensor([0] + np.cumsum(lengths).tolist(), dtype=torch.int32, device="cuda")
    k, v = (torch.empty(n, hkv, dim, device="cuda") for _ in range(2))
    sffn.sffn_kv_gather(cache.handle, sffn.KvBatch(table, kv_len, start, n), k, v)
    cache.check_error()
    both = torch.stack((k, v), 1)
    return [both[a:b].clone() for a, b in zip(start.tolist(), start.tolist()[1:])]


@pytest.mark.parametrize("place", ["in place", "another table"])
@pytest.mark.parametrize("layers,groups,beams,page,hkv,dim,group,lengths", [
    (1, 1, 4, 16, 8, 128, 128, [37]), (3, 2, 2, 32, 3, 64, 32, [64, 5]), (2, 3, 5, 64, 1, 256, 64, [63, 129, 65]),
    (1, 2, 1, 16, 2, 128, 64, [16, 17]), (2, 1, 16, 16, 4, 64, 64, [15]), (1, 1, 64, 16, 2, 64, 32, [23]),
    (1, 3, 3, 32, 2, 128, 32, [0, 1, 32]), (1, 1, 3, 16, 40, 256, 32, [30])])
def test_reorder(sffn, place, layers, groups, beams, page, hkv, dim, group, lengths):
    n_seq, per = groups * beams, [n for n in lengths for _ in range(beams)]
    width = max(1, -(-max(lengths) // page) + 1)
    caches, table = make_caches(sffn, layers, n_seq, width, page, hkv, dim, group)
    kv_len = fill(sffn, caches, table, per, hkv, dim)
    before = [read(sffn, c, table, per, hkv, dim) for c in caches]
    old = table.clone()
    parent = torch.randint(0, beams, (groups, beams), generator=gen(9), device="cuda", dtype=torch.int32)
    if beams > 1:
        parent[0, :2] = torch.tensor([1, 0], device="cuda", dtype=torch.int32)    # two sequences that swap
    if place == "in place":
        out = table
    else:
        # every sequence's next page, which nothing else names, is its last one in the other table
        out = torch.full((n_seq, width + 2), -5, dtype=torch.int32, device="cuda")
        for s, n in enumerate(per):
            out[s, n // page] = old[s, width - 1]
        out = out[:, :width]
    kept = out.clone()
    sffn.sffn_kv_reorder(sffn.KvCaches(caches), sffn.KvBatch(table, kv_len), parent.flatten(), beams, out)
    for c in caches:
        c.check_error()
    want = kept.clone()
    source = [s // beams * beams + int(parent.flatten()[s]) for s in range(n_seq)]
    for s, m in enumerate(source):
        want[s, :per[s] // page] = old[m, :per[s] // page]
    assert torch.equal(out, want)
    if place != "in place":
        assert torch.equal(table, old)
    for c, was in zip(caches, before):
        now = read(sffn, c, out.contiguous(), per, hkv, dim)
        for s, m in enumerate(source):
            assert (now[s] is None and was[m] is None) or torch.equal(now[s], was[m])


def test_reorder_then_append_keeps_copies_apart(sffn):
    """Sequences that go on as copies of one write their next positions without reaching each other's."""
    beams, page, hkv, dim, n = 4, 16, 2, 64, 29
    caches, table = make_caches(sffn, 2, beams, 4, page, hkv, dim, 64)
    kv_len = fill(sffn, caches, table, [n] * beams, hkv, dim)
    batch = sffn.KvBatch(table, kv_len)
    rows = [read(sffn, c, table, [n] * beams, hkv, dim) for c in caches]
    g = gen(5)
    for step in range(24):                                      # past two page ends
        parent = torch.randint(0, beams, (beams,), generator=g, device="cuda", dtype=torch.int32)
        sffn.sffn_kv_reorder(sffn.KvCaches(caches), batch, parent, beams)
        kv_len += 1
        for c, held in zip(caches, rows):
            k, v = (torch.randn(beams, hkv, dim, generator=g, device="cuda") for _ in range(2))
            sffn.sffn_kv_append(c.handle, batch, None, k, v)
            last = [r[-1:] for r in read(sffn, c, table, [n + step + 1] * beams, hkv, dim)]
            held[:] = [torch.cat((held[int(parent[s])], last[s])) for s in range(beams)]
    for c, held in zip(caches, rows):
        now = read(sffn, c, table, [n + 24] * beams, hkv, dim)
        assert all(torch.equal(a, b) for a, b in zip(now, held))
        c.check_error()


def test_reorder_leaves_a_group_with_faults(sffn):
    beams, page, hkv, dim = 3, 16, 2, 64
    per = [20] * 3 + [21] * 3 + [22] * 3
    for fault in ("parent", "negative parent", "length", "too long", "page"):
        caches, table = make_caches(sffn, 1, 9, 2, page, hkv, dim, 32)
        kv_len = fill(sffn, caches, table, per, hkv, dim)
        parent = torch.tensor([1, 2, 0] * 3, dtype=torch.int32, device="cuda")
        was = read(sffn, caches[0], table, per, hkv, dim)
        old = table.clone()
        if fault.endswith("parent"):
            parent[4] = -1 if fault[0] == "n" else 3
        elif fault == "length":
            kv_len[5] = 22
        elif fault == "too long":
            kv_len[3:6] = 33
        else:
            table[3, 1] = 18                                    # sequence 4 has its last page there
        sffn.sffn_kv_reorder(sffn.KvCaches(caches), sffn.KvBatch(table, kv_len), parent, beams)
        with pytest.raises(sffn.SffnError):
            caches[0].check_error()
        now = read(sffn, caches[0], old if fault == "page" else table, per, hkv, dim)
        for s in range(9):
            m = s // 3 * 3 + (s % 3 + 1) % 3
            if fault == "page":
                continue                                        # the bad page is neither read nor written
            assert torch.equal(now[s], was[s] if s // 3 == 1 else was[m]), fault
        if fault != "page":
            assert torch.equal(table[3:6], old[3:6])
        else:
            # sequences 3 and 5 copy from 4 and 3: 3 has no page to copy to, 5 none to copy from
            assert torch.equal(now[3][16:], was[3][16:]) and torch.equal(now[5][16:], was[5][16:])
            assert torch.equal(now[4][16:], was[5][16:])


def test_reorder_refusals(sffn):
    caches, table = make_caches(sffn, 1, 4, 2, 16, 2, 64, 32)
    other = sffn.KvCache(8, 16, 2, 64, 64)
    kv_len = torch.full((4,), 5, dtype=torch.int32, device="cuda")
    parent, batch = torch.zeros(4, dtype=torch.int32, device="cuda"), sffn.KvBatch(table, kv_len)
    one = sffn.KvCaches(caches)
    wide = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    held = sffn.KvBatch(wide[:4], kv_len)
    for bad in (lambda: sffn.sffn_kv_reorder(sffn.KvCaches([caches[0], other]), batch, parent, 4),
                lambda: sffn.sffn_kv_reorder(sffn.KvCaches([caches[0], caches[0]]), batch, parent, 4),
                lambda: sffn.sffn_kv_reorder(sffn.KvCaches([]), batch, parent, 4),
                lambda: sffn.sffn_kv_reorder(one, batch, parent, 3),
                lambda: sffn.sffn_kv_reorder(one, batch, parent, 0),
                lambda: sffn.sffn_kv_reorder(one, batch, parent, 65),
                lambda: sffn.sffn_kv_reorder(one, held, parent, 4, wide[1:])):         # overlaps the table
        with pytest.raises(sffn.SffnError):
            bad()
    for bad in (lambda: sffn.sffn_kv_reorder(one, batch, parent[:3], 4),
                lambda: sffn.sffn_kv_reorder(one, batch, parent.long(), 4),
                lambda: sffn.sffn_kv_reorder(one, batch, parent, 4, table[:, :1])):
        with pytest.raises(ValueError):
            bad()
    caches[0].check_error()
