"""The attention half of a decode step on the GPU against the plain
implementations of attn_ref: 4-bit projections, the append to the paged 4-bit
cache, the attention over it, and the three together."""

import math

import numpy as np
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


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


def host(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ projections

def make_linear(sffn, n, k, group, seed, zeros, bias, sdtype="f16", max_batch=32):
    g = gen(seed)
    codes = torch.randint(-8, 8, (n, k), generator=g, device="cuda", dtype=torch.int8)
    scales = (0.02 + 0.05 * torch.rand(n, k // group, generator=g, device="cuda")).to(TORCH[sdtype])
    z = torch.randint(-8, 8, scales.shape, generator=g, device="cuda").to(TORCH[sdtype]) if zeros else None
    b = torch.randn(n, generator=g, device="cuda") if bias else None
    return sffn.Linear.from_weights(codes, scales, z, b, max_batch=max_batch), codes, scales, z, b


def check_linear(sffn, n, k, group, B, dtype, zeros=False, bias=False, residual=False, sdtype="f16", seed=0, x=None):
    lin, codes, scales, z, b = make_linear(sffn, n, k, group, seed, zeros, bias, sdtype)
    g = gen(seed + 1)
    if x is None:
        x = torch.randn(B, k, generator=g, device="cuda")
        x[:, :: max(1, k // 5)] *= 30.0
        x = x.to(TORCH[dtype])
    r = torch.randn(B, n, generator=g, device="cuda").to(TORCH[dtype]) if residual else None
    y = torch.full((B, n), float("nan"), device="cuda", dtype=TORCH[dtype])
    sffn.sffn_linear_forward(lin.handle, x, y, r, lin.workspace(B))
    want, tol = R.linear(host(x), codes.cpu().numpy(), host(scales), None if z is None else host(z),
                         None if b is None else host(b), None if r is None else host(r), group)
    R.assert_close(host(y), want, tol, dtype, f"linear {n}x{k} G{group} B{B} {dtype}")
    lin.check_error()
    return lin, x, y, r


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_linear_types_and_groups(sffn, dtype, group, zeros):
    check_linear(sffn, 200, 896, group, 3, dtype, zeros=zeros, bias=True, residual=True, seed=group)


@pytest.mark.parametrize("B", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 24, 31, 32])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_batches(sffn, B, dtype):
    check_linear(sffn, 333, 1280, 64, B, dtype, residual=B % 2 == 0, zeros=B % 3 == 0, seed=B)


@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (15, 96, 32), (16, 64, 64), (17, 128, 128), (1, 8192, 128),
                                       (4097, 160, 32), (5, 11008, 32), (2432, 2432, 64), (31, 65536, 128),
                                       (10240, 640, 128)])
@pytest.mark.parametrize("B", [1, 6, 32])
def test_linear_shapes(sffn, n, k, group, B):
    check_linear(sffn, n, k, group, B, "f32", seed=n + k, zeros=n % 2 == 1, bias=True)


@pytest.mark.parametrize("sdtype", ["f32", "f16", "bf16"])
def test_linear_scale_types(sffn, sdtype):
    check_linear(sffn, 100, 512, 32, 2, "f32", zeros=True, sdtype=sdtype, seed=5)


def test_linear_range_of_inputs(sffn):
    """Tokens of very small and very large numbers, a zero token, and one huge element."""
    x = torch.randn(6, 1024, generator=gen(3), device="cuda")
    x[0] *= 1e-30
    x[1] *= 1e30
    x[2] = 0
    x[3, 17] = 1e6
    x[4] *= torch.logspace(-12, 3, 1024, device="cuda")
    x[5] = 2.0 ** -126
    check_linear(sffn, 64, 1024, 128, 6, "f32", x=x, seed=9)


def test_linear_strides_in_place_residual_and_untouched_rows(sffn):
    lin, codes, scales, z, b = make_linear(sffn, 77, 256, 64, 1, False, False)
    g = gen(2)
    xs = torch.randn(5, 3, 256 + 8, generator=g, device="cuda")
    x = xs[:, 1, :256]
    ys = torch.randn(5, 2, 91, generator=g, device="cuda")
    before = ys.clone()
    y = ys[:, 1, 7:84]                       # odd stride, odd offset
    sffn.sffn_linear_forward(lin.handle, x, y, y, lin.workspace(5))
    want, tol = R.linear(host(x), codes.cpu().numpy(), host(scales), None, None, host(before[:, 1, 7:84]), 64)
    R.assert_close(host(y), want, tol, "f32", "strided, in place")
    ys[:, 1, 7:84] = before[:, 1, 7:84]
    assert torch.equal(ys, before)


def test_linear_non_finite_tokens_stay_apart(sffn):
    lin, x, y, _ = check_linear(sffn, 130, 512, 64, 5, "f32", zeros=True, seed=4)
    x = x.clone()
    x[1, 100] = float("nan")
    x[3, 5] = float("inf")
    z = torch.empty_like(y)
    sffn.sffn_linear_forward(lin.handle, x, z, None, lin.workspace(5))
    assert not z[[1, 3]].isfinite().any()
    assert torch.equal(z[[0, 2, 4]], y[[0, 2, 4]])


def test_linear_same_bits_on_other_streams_and_in_graphs(sffn):
    lin, x, y, r = check_linear(sffn, 1000, 4096, 128, 2, "f32", residual=True, seed=6)
    ws, z = lin.workspace(2), torch.empty_like(y)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(3):
            sffn.sffn_linear_forward(lin.handle, x, z, r, ws)
    st.synchronize()
    assert torch.equal(z, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sffn.sffn_linear_forward(lin.handle, x, z, r, ws)
    z.zero_()
    graph.replay()
    assert torch.equal(z, y)


def test_linear_refuses_bad_codes(sffn):
    codes = torch.zeros(8, 64, dtype=torch.int8, device="cuda")
    scales = torch.ones(8, 2, dtype=torch.float16, device="cuda")
    lin = sffn.Linear(64, 8, 32)
    x, y = torch.zeros(1, 64, device="cuda"), torch.zeros(1, 8, device="cuda")
    with pytest.raises(sffn.SffnError) as e:
        sffn.sffn_linear_forward(lin.handle, x, y, None, lin.workspace())
    assert e.value.status == sffn.SFFN_ERR_INVALID_ARG
    codes[7, 63] = 8
    with pytest.raises(sffn.SffnError) as e:
        sffn.sffn_linear_pack(lin.handle, codes, scales)
    assert e.value.status == sffn.SFFN_ERR_DEVICE
    with pytest.raises(sffn.SffnError):
        sffn.sffn_linear_forward(lin.handle, x, y, None, lin.workspace())
    codes[7, 63] = 7
    sffn.sffn_linear_pack(lin.handle, codes, scales)
    sffn.sffn_linear_forward(lin.handle, x, y, None, lin.workspace())
    with pytest.raises(sffn.SffnError):
        sffn.sffn_linear_forward(lin.handle, torch.zeros(2, 64, device="cuda"), torch.zeros(2, 8, device="cuda"))
    with pytest.raises(sffn.SffnError):
        sffn.sffn_linear_forward(lin.handle, torch.zeros(65, device="cuda")[1:].view(1, 64), y)
    with pytest.raises(ValueError):
        sffn.sffn_linear_forward(lin.handle, x, y.half())
    with pytest.raises(ValueError):
        sffn.sffn_linear_forward(lin.handle, x, y, y.view(8, 1))


# ------------------------------------------------------------------ cache

class Case:
    """Sequences in a paged cache with shuffled pages; lens: (cached, new) each."""

    def __init__(self, sffn, lens, hkv, D, G, P, dtype="f32", seed=0, spare=2, fill=None, extra_pages=0):
        self.lens, self.hkv, self.D, self.G, self.P, self.dtype = lens, hkv, D, G, P, TORCH[dtype]
        self.g = gen(seed)
        width = max(1, max(-(-n // P) for n, _ in lens)) + 1
        self.n_pages = len(lens) * width + spare + extra_pages
        self.cache = sffn.KvCache(self.n_pages, P, hkv, D, G)
        order = torch.randperm(len(lens) * width + spare, generator=self.g, device="cuda")[: len(lens) * width]
        self.table = (order + extra_pages).view(len(lens), width).to(torch.int32)
        self.kv_len = torch.tensor([n for n, _ in lens], dtype=torch.int32, device="cuda")
        self.total, self.fresh = sum(n for n, _ in lens), sum(q for _, q in lens)
        self.all = sffn.KvBatch(self.table, self.kv_len, self.starts([n for n, _ in lens]), self.total)
        self.new = sffn.KvBatch(self.table, self.kv_len, self.starts([q for _, q in lens]), self.fresh)

    def starts(self, counts):
        return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(self.dtype)

    def fill_cache(self, sffn, spread=1.0):
        k = self.randn(self.total, self.hkv, self.D) * spread + torch.linspace(-1, 1, self.D, device="cuda").to(self.dtype)
        v = self.randn(self.total, self.hkv, self.D)
        sffn.sffn_kv_append(self.cache.handle, self.all, None, k, v)
        self.k, self.v = (R.stored(t.float().cpu().numpy(), self.G) for t in (k, v))
        step, mid, _ = R.group_params(k.float().cpu().numpy(), self.G)
        self.ksize = np.repeat(abs(mid.astype(np.float64)) + (15 if self.dtype == torch.float32 else 30) * step.astype(np.float64), self.G, axis=-1)
        mid = R.group_params(v.float().cpu().numpy(), self.G)[1].astype(np.float64)
        self.vsize = None if self.dtype == torch.float32 else abs(self.v) + np.repeat(abs(mid), self.G, axis=-1)
        return k, v


SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("P", [16, 32, 64])
def test_append_holds_the_rounded_rows(sffn, D, G, P):
    c = Case(sffn, [(1, 1), (70, 70), (0, 0), (33, 33)], 3, D, G, P, seed=D + G + P)
    k, v = c.fill_cache(sffn)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    sffn.sffn_kv_gather(c.cache.handle, c.all, ko, vo)
    assert np.array_equal(ko.cpu().numpy(), c.k) and np.array_equal(vo.cpu().numpy(), c.v)
    # the last two positions of every sequence, one output only
    lens = [(n, min(n, 2)) for n, _ in c.lens]
    b = sffn.KvBatch(c.table, c.kv_len, c.starts([q for _, q in lens]), sum(q for _, q in lens))
    part = torch.empty(sum(q for _, q in lens), 3, D, device="cuda")
    sffn.sffn_kv_gather(c.cache.handle, b, None, part)
    ends = np.cumsum([n for n, _ in lens])
    want = np.concatenate([c.v[e - q:e] for e, (_, q) in zip(ends, lens)])
    assert np.array_equal(part.cpu().numpy(), want)
    c.cache.check_error()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("D,G,R_dim", [(64, 32, 64), (128, 128, 128), (128, 64, 32), (256, 128, 256), (256, 64, 6)])
def test_append_rotates(sffn, dtype, style, D, G, R_dim):
    lens, hq, hkv = [(5, 2), (40, 17), (1, 1)], 6, 2
    c = Case(sffn, lens, hkv, D, G, 16, dtype, seed=D + R_dim)
    rope = sffn.Rope.of_base(64, R_dim, style=style)
    # queries, keys and values as views of one array, queries turned in place
    qkv = c.randn(c.fresh, hq + 2 * hkv, D)
    q, k, v = qkv.split((hq, hkv, hkv), 1)
    f = qkv.float().cpu().numpy()
    pos = np.concatenate([np.arange(n - m, n) for n, m in lens])
    turned = R.rotate(f[:, :hq + hkv], rope.table.cpu().numpy()[pos], style)
    sffn.sffn_kv_append(c.cache.handle, c.new, q, k, v, q, rope)
    ko, vo = (torch.empty(c.fresh, hkv, D, device="cuda") for _ in range(2))
    sffn.sffn_kv_gather(c.cache.handle, c.new, ko, vo)
    assert torch.equal(q.cpu(), torch.from_numpy(turned[:, :hq]).to(TORCH[dtype]))
    assert torch.equal(k.float().cpu(), torch.from_numpy(f[:, hq:hq + hkv]))          # inputs untouched
    assert np.array_equal(ko.cpu().numpy(), R.stored(turned[:, hq:], G))
    assert np.array_equal(vo.cpu().numpy(), R.stored(f[:, hq + hkv:], G))
    c.cache.check_error()


def test_append_with_given_positions_and_rows_without_a_place(sffn):
    """Three rows for a sequence of length one: two have no place, their queries are still turned by their positions."""
    c = Case(sffn, [(1, 3), (2, 2)], 1, 64, 64, 16, seed=1)
    pos = torch.tensor([7, 0, 9, 3, 3], dtype=torch.int32, device="cuda")
    base = sffn.Rope.of_base(10, 64)
    rope = sffn.Rope(base.table, "halves", pos)
    q, k, v = (c.randn(5, 1, 64) for _ in range(3))
    qo = torch.empty_like(q)
    sffn.sffn_kv_append(c.cache.handle, c.new, q, k, v, qo, rope)
    cs = base.table.cpu().numpy()[pos.cpu().numpy()]
    assert np.array_equal(qo.cpu().numpy(), R.rotate(q.cpu().numpy(), cs, "halves"))
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    sffn.sffn_kv_gather(c.cache.handle, c.new, ko, vo)
    want = R.stored(R.rotate(k.cpu().numpy(), cs, "halves"), 64)
    want[:2] = 0
    assert np.array_equal(ko.cpu().numpy(), want)
    c.cache.check_error()
    sffn.sffn_kv_append(c.cache.handle, c.new, q, k, v, qo, sffn.Rope(base.table[:9].contiguous(), "halves", pos))
    with pytest.raises(sffn.SffnError) as e:
        c.cache.check_error()
    assert e.value.status == sffn.SFFN_ERR_DEVICE
    assert torch.equal(qo[2], q[2])


def test_append_extreme_rows(sffn):
    """Constant, zero, tiny, huge and non-finite groups."""
    c = Case(sffn, [(8, 8)], 1, 128, 64, 16, seed=2)
    k = c.randn(8, 1, 128)
    k[0] = 3.25
    k[1] = 0
    k[2] *= 1e-7
    k[3] *= 1e5
    k[4, 0, 3] = float("inf")
    k[5, 0, 100] = float("nan")
    k[6] = -1e30
    k[7, 0, :64] = 1e-30
    sffn.sffn_kv_append(c.cache.handle, c.new, None, k, k)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    sffn.sffn_kv_gather(c.cache.handle, c.new, ko, vo)
    want = R.stored(k.cpu().numpy(), 64)
    assert np.array_equal(ko.cpu().numpy(), want, equal_nan=True) and np.array_equal(vo.cpu().numpy(), want, equal_nan=True)
    assert np.isnan(want[4, 0, :64]).all() and np.isfinite(want[4, 0, 64:]).all() and np.isnan(want[5, 0, 64:]).all()
    c.cache.check_error()


def test_bad_pages_and_lengths_are_flagged(sffn):
    c = Case(sffn, [(40, 40), (20, 20)], 2, 64, 64, 16, seed=3)
    k, v = c.fill_cache(sffn)
    c.cache.check_error()
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    good = c.table.clone()
    for bad in (-1, c.n_pages, 2 ** 31 - 1):
        c.table[0, 1] = bad
        sffn.sffn_kv_append(c.cache.handle, c.all, None, k + 1, v)
        with pytest.raises(sffn.SffnError):
            c.cache.check_error()
        c.cache.check_error()                                    # cleared
        sffn.sffn_kv_append(c.cache.handle, c.all, None, k, v)   # the good pages hold the old rows again
        with pytest.raises(sffn.SffnError):
            c.cache.check_error()
        c.table.copy_(good)
        sffn.sffn_kv_gather(c.cache.handle, c.all, ko, vo)
        assert np.array_equal(ko.cpu().numpy(), c.k)             # nothing else was written
        c.cache.check_error()
        c.table[0, 1] = bad
        q, out = c.randn(60, 2, 64), torch.empty(60, 2, 64, device="cuda")
        sffn.sffn_attend(c.cache.handle, c.all, q, out, None, 0.1, 0, c.cache.workspace(c.all, 2))
        with pytest.raises(sffn.SffnError):
            c.cache.check_error()
        c.table.copy_(good)
    for n in (c.table.shape[1] * 16 + 1, 2 ** 31 - 1, -5):
        c.kv_len[1] = n
        sffn.sffn_kv_gather(c.cache.handle, c.new, ko, vo)
        with pytest.raises(sffn.SffnError):
            c.cache.check_error()


# ------------------------------------------------------------------ attention

def check_attention(sffn, lens, hq, hkv, D, G, P, dtype="f32", window=0, scale=None, seed=0, spread=1.0, sharp=1.0,
                    case=None, with_lse=True):
    c = case or Case(sffn, lens, hkv, D, G, P, dtype, seed)
    if case is None:
        c.fill_cache(sffn, spread)
    scale = sharp / math.sqrt(D) if scale is None else scale
    q = c.randn(c.fresh, hq, D)
    out = torch.full_like(q, float("nan"))
    lse = torch.full((c.fresh, hq), float("nan"), device="cuda") if with_lse else None
    sffn.sffn_attend(c.cache.handle, c.new, q, out, lse, scale, window, c.cache.workspace(c.new, hq))
    qh, oh = host(q), host(out)
    at = row = 0
    for n, m in lens:
        want, wlse, tol = R.attention(qh[row:row + m], c.k[at:at + n], c.v[at:at + n], m, scale, window, c.ksize[at:at + n],
                                      None if c.vsize is None else c.vsize[at:at + n])
        R.assert_close(oh[row:row + m], want, tol, dtype, f"attention len {n} new {m}")
        if with_lse:
            got = lse[row:row + m].double().cpu().numpy()
            empty = np.isinf(wlse)
            assert np.array_equal(np.isneginf(got), empty)
            got, wlse = got[~empty], wlse[~empty]
            assert (np.abs(got - wlse) <= 2e-5 * np.maximum(1, np.abs(wlse))).all()
        at, row = at + n, row + m
    c.cache.check_error()
    return c, q, out, lse


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_attention_shapes_and_types(sffn, D, G, dtype):
    check_attention(sffn, [(97, 1), (1, 1), (300, 3)], 6, 2, D, G, 16 if D == 64 else 32, dtype, seed=D + G)


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 1000, 4097])
def test_attention_lengths(sffn, n, P):
    check_attention(sffn, [(n, 1)], 8, 1, 128, 128, P, seed=n + P)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 7), (4, 2), (5, 1), (16, 2), (9, 1), (40, 8), (71, 1)])
def test_attention_head_ratios(sffn, hq, hkv):
    check_attention(sffn, [(130, 1), (77, 2)], hq, hkv, 64, 32, 16, seed=hq)


@pytest.mark.parametrize("window", [1, 2, 31, 64, 65, 100, 1000, 2 ** 31 - 1])
def test_attention_windows(sffn, window):
    check_attention(sffn, [(300, 1), (70, 33), (64, 64), (5, 5)], 4, 2, 128, 64, 16, window=window, seed=window % 97)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_rows_that_see_nothing(sffn, dtype):
    """Empty sequences, sequences without rows, and more rows than cached positions."""
    check_attention(sffn, [(0, 1), (3, 7), (0, 0), (40, 0), (0, 5), (65, 66)], 4, 2, 128, 128, 16, dtype, seed=11)


def test_attention_one_token_per_sequence_without_starts(sffn):
    c = Case(sffn, [(n, 1) for n in (5, 0, 64, 129)], 2, 64, 64, 32, seed=12)
    c.fill_cache(sffn)
    _, q, out, lse = check_attention(sffn, c.lens, 8, 2, 64, 64, 32, case=c)
    b = sffn.KvBatch(c.table, c.kv_len)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    sffn.sffn_attend(c.cache.handle, b, q, o2, l2, 1 / 8, 0, c.cache.workspace(b, 8))
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("sharp", [0.0, 1e-3, 30.0, -5.0])
def test_attention_flat_and_sharp(sffn, sharp):
    check_attention(sffn, [(2500, 2)], 8, 2, 128, 64, 64, sharp=sharp, seed=13)


def test_attention_many_sequences(sffn):
    lens = [((37 * i) % 211, (i % 4)) for i in range(150)]
    check_attention(sffn, lens, 4, 2, 64, 64, 16, seed=14)


def test_attention_many_rows_a_sequence(sffn):
    check_attention(sffn, [(200, 200), (150, 90)], 8, 2, 64, 64, 16, "f16", seed=15)


def test_attention_long(sffn):
    check_attention(sffn, [(30011, 1), (9, 1)], 8, 1, 128, 128, 64, seed=16)


def test_attention_far_pages(sffn):
    """Pages whose byte offset passes 32 bits."""
    block = 64 * (128 + 8)
    pages = (5 << 30) // (block * 8)
    c = Case(sffn, [(300, 1), (65, 2)], 8, 128, 128, 64, seed=17, extra_pages=pages)
    assert c.n_pages * block * 8 > 5 << 30
    k, v = c.fill_cache(sffn)
    check_attention(sffn, c.lens, 16, 8, 128, 128, 64, case=c)


def poison(sffn, c):
    """Every slot of every page holds NaN groups."""
    rows = c.n_pages * c.P
    table = torch.arange(c.n_pages, device="cuda", dtype=torch.int32)[None]
    b = sffn.KvBatch(table, torch.tensor([rows], dtype=torch.int32, device="cuda"),
                     torch.tensor([0, rows], dtype=torch.int32, device="cuda"), rows)
    bad = torch.full((rows, c.hkv, c.D), float("nan"), device="cuda", dtype=c.dtype)
    sffn.sffn_kv_append(c.cache.handle, b, None, bad, bad)


@pytest.mark.parametrize("P", [16, 64])
def test_attention_never_uses_what_it_does_not_see(sffn, P):
    """Slots past the end, and positions outside the window or after the row, hold NaN."""
    lens = [(65, 2), (1, 1), (31, 3), (130, 1)]
    c = Case(sffn, lens, 2, 128, 32, P, seed=18)
    poison(sffn, c)
    c.fill_cache(sffn)
    check_attention(sffn, lens, 8, 2, 128, 32, P, case=c)
    # position 50 of the first sequence is NaN: rows whose window starts after it are as before
    at = sffn.KvBatch(c.table[:1].contiguous(), torch.tensor([51], dtype=torch.int32, device="cuda"))
    nan = torch.full((1, 2, 128), float("nan"), device="cuda")
    q = c.randn(c.fresh, 8, 128)
    ws = c.cache.workspace(c.new, 8)
    outs = []
    for poisoned in (False, True):
        if poisoned:
            sffn.sffn_kv_append(c.cache.handle, at, None, nan, nan)
        out, lse = torch.empty_like(q), torch.empty(c.fresh, 8, device="cuda")
        sffn.sffn_attend(c.cache.handle, c.new, q, out, lse, 0.1, 14, ws)
        outs.append((out, lse))
    (a, la), (b, lb) = outs
    # rows at positions 63 and 64 see 50..63 and 51..64
    assert b[0].isnan().all() and lb[0].isnan().all()
    assert torch.equal(a[1:], b[1:]) and torch.equal(la[1:], lb[1:])


def test_attention_non_finite_query_rows_stay_apart(sffn):
    c, q, out, lse = check_attention(sffn, [(100, 3)], 8, 2, 64, 64, 16, seed=19)
    q2 = q.clone()
    q2[1, 3, 5] = float("nan")
    q2[2, 6, 0] = float("inf")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    sffn.sffn_attend(c.cache.handle, c.new, q2, o2, l2, 1 / 8, 0, c.cache.workspace(c.new, 8))
    bad = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[2, 6] = True
    assert o2[bad].isnan().all()
    assert torch.equal(o2[~bad], out[~bad]) and torch.equal(l2[~bad], lse[~bad])


def test_attention_strided_rows_streams_and_graphs(sffn):
    c, q, out, lse = check_attention(sffn, [(700, 1), (1300, 2), (3, 1)], 8, 2, 128, 128, 16, seed=20)
    wide = torch.randn(c.fresh, 12, 136, device="cuda")
    qs = wide[:, 2:10, :128]
    qs.copy_(q)
    os = torch.empty(8, c.fresh, 128, device="cuda").transpose(0, 1)
    l2, ws, scale = torch.empty_like(lse), c.cache.workspace(c.new, 8), 1 / math.sqrt(128)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(3):
            sffn.sffn_attend(c.cache.handle, c.new, qs, os, l2, scale, 0, ws)
    st.synchronize()
    assert torch.equal(os, out) and torch.equal(l2, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sffn.sffn_attend(c.cache.handle, c.new, qs, os, l2, scale, 0, ws)
    c.kv_len[1] -= 700                                   # lengths are read at every replay
    graph.replay()
    ref, rl = torch.empty_like(out), torch.empty_like(lse)
    sffn.sffn_attend(c.cache.handle, c.new, q, ref, rl, scale, 0, ws)
    assert torch.equal(os, ref) and torch.equal(l2, rl) and not torch.equal(ref[1], out[1])


def test_no_tokens(sffn):
    c = Case(sffn, [(5, 0)], 2, 64, 64, 16)
    e = torch.empty(0, 2, 64, device="cuda")
    sffn.sffn_kv_append(c.cache.handle, c.new, e, e, e, e)
    sffn.sffn_kv_gather(c.cache.handle, c.new, e, e)
    sffn.sffn_attend(c.cache.handle, c.new, e, e, None, 1.0, 0, c.cache.workspace(c.new, 2))
    c.cache.check_error()


def test_attention_refusals(sffn):
    c = Case(sffn, [(5, 1)], 2, 64, 64, 16)
    q = torch.zeros(1, 4, 64, device="cuda")
    out, ws = torch.empty_like(q), c.cache.workspace(c.new, 4)
    h = c.cache.handle
    for call in (
        lambda: sffn.sffn_attend(h, c.new, q[:, :3], out[:, :3], None, 1.0, 0, ws),            # heads
        lambda: sffn.sffn_attend(h, c.new, q, out, None, float("nan"), 0, ws),
        lambda: sffn.sffn_attend(h, c.new, q, out, None, 1.0, -1, ws),
        lambda: sffn.sffn_attend(h, c.new, torch.zeros(257, device="cuda")[1:].view(1, 4, 64), out, None, 1.0, 0, ws),
        lambda: sffn.sffn_kv_append(h, c.new, None, torch.zeros(1, 2, 66, device="cuda")[..., :64].transpose(0, 0)[:, :, :64],
                                    torch.zeros(1, 2, 66, device="cuda")[..., :64]),            # head stride 66
    ):
        with pytest.raises(sffn.SffnError) as e:
            call()
        assert e.value.status == sffn.SFFN_ERR_INVALID_ARG
    for call in (
        lambda: sffn.sffn_attend(h, c.new, q, out.half(), None, 1.0, 0, ws),
        lambda: sffn.sffn_attend(h, c.new, q.expand(2, 4, 64), out, None, 1.0, 0, ws),
        lambda: sffn.sffn_kv_append(h, c.new, None, out[:, :2], out[:, :2].half()),
        lambda: sffn.KvBatch(c.table.long(), c.kv_len),
        lambda: sffn.KvBatch(c.table, c.kv_len, c.new.q_start),
        lambda: sffn.Rope(torch.zeros(4, 2, device="cuda")),
    ):
        with pytest.raises(ValueError):
            call()


def test_attention_workspace_comes_with_any_contents(sffn):
    """Items cut by the borders of blocks, with the workspace full of ones, of noise, and of what a call left there."""
    lens = [(5000, 1), (70, 2), (1700, 1), (64, 1), (65, 1)]
    c, q, out, lse = check_attention(sffn, lens, 8, 2, 128, 64, 32, seed=21)
    ws, scale = c.cache.workspace(c.new, 8), 1 / math.sqrt(128)
    for fill in (lambda: ws.fill_(255), lambda: ws.random_(0, 256, generator=c.g), lambda: None, lambda: ws.zero_(), lambda: None):
        fill()
        o2, l2 = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
        sffn.sffn_attend(c.cache.handle, c.new, q, o2, l2, scale, 0, ws)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("seqs,hkv", [(1, 1), (2, 1), (1, 8), (3, 5), (40, 8)])
@pytest.mark.parametrize("n", [64, 150, 9000])
def test_attention_cuts(sffn, seqs, hkv, n):
    """From fewer units than blocks to many, whatever the borders cut; equal bits at every call."""
    n = n if seqs * hkv < 100 else min(n, 700)
    c, q, out, lse = check_attention(sffn, [(n + 3 * s, 1) for s in range(seqs)], 2 * hkv, hkv, 64, 64, 64, seed=n + seqs)
    ws = c.cache.workspace(c.new, 2 * hkv)
    for _ in range(20):
        o2, l2 = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
        sffn.sffn_attend(c.cache.handle, c.new, q, o2, l2, 1 / 8, 0, ws)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("hkv", [1, 5])
@pytest.mark.parametrize("first", [(9000, 1), (64 * 15, 1), (64 * 17, 2), (64 * 33, 1)])
def test_attention_short_and_long_histories_in_one_call(sffn, first, hkv, dtype):
    """Blocks of work begin and end between short histories, within long ones, and where one follows the other."""
    lens = [first, (500, 1), (1, 1), (4000, 1), (70, 3), (0, 1), (2000, 1), (0, 0), (64 * 16, 1), (64 * 32, 1), (12000, 1),
            (64, 64), (1500, 1)]
    check_attention(sffn, lens, 2 * hkv, hkv, 128, 128, 64, dtype, seed=first[0] + hkv)


@pytest.mark.parametrize("seqs", [3, 40])
def test_attention_refuses_rows_that_lie_in_several_sequences(sffn, seqs):
    """Row starts that descend set the error word; nothing is written, and the cache works on."""
    c = Case(sffn, [(64, 2)] * seqs, 2, 64, 64, 16)
    c.fill_cache(sffn, 1.0)
    q = c.randn(c.fresh, 4, 64)
    out = torch.full_like(q, 7.0)
    ws = c.cache.workspace(c.new, 4)
    starts = c.new.q_start.clone()
    c.new.q_start[seqs - 1] = 0
    sffn.sffn_attend(c.cache.handle, c.new, q, out, None, 1.0, 0, ws)
    with pytest.raises(sffn.SffnError):
        c.cache.check_error()
    assert (out == 7.0).all()
    c.new.q_start.copy_(starts)
    check_attention(sffn, [(64, 2)] * seqs, 4, 2, 64, 64, 16, case=c)
