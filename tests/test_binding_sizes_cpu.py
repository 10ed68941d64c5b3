"""The binding compares a call's tensors with the sizes of its handle before the
C call, which sees pointers and strides only: with one row it could not tell a
short array. No GPU: the library is replaced by one that counts calls."""

import types

import pytest
import torch


@pytest.fixture()
def lib(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    from activation_sparse_ffn_gb300 import sffn
    calls = []

    def take(name, result=0):
        def f(*args):
            calls.append(name)
            return result
        return f

    def create(handle):
        def f(desc, out):
            out._obj.value = handle
            return 0
        return f

    def get_desc(made):
        def f(handle, out):
            for n, _ in out._obj._fields_:
                setattr(out._obj, n, getattr(made[handle], n))
            return 0
        return f

    linear, kv = sffn.make_linear_desc(256, 96, 64, "f16", max_batch=4), sffn.make_kv_desc(4, 16, 3, 64, 32)
    fake = types.SimpleNamespace(
        sffn_linear_create=create(4096), sffn_kv_create=create(8192),
        sffn_linear_get_desc=get_desc({4096: linear}), sffn_kv_get_desc=get_desc({8192: kv}),
        **{n: take(n) for n in ("sffn_linear_forward", "sffn_linear_pack", "sffn_linear_destroy", "sffn_kv_append",
                                "sffn_kv_gather", "sffn_attend", "sffn_kv_destroy")})
    monkeypatch.setattr(sffn, "_lib", fake)
    monkeypatch.setattr(sffn, "_stream", lambda stream: None)
    sffn.calls = calls
    h = sffn.sffn_linear_create(linear)
    c = sffn.sffn_kv_create(kv)
    yield sffn, h, c
    sffn.sffn_linear_destroy(h)
    sffn.sffn_kv_destroy(c)
    del sffn.calls


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("B", [1, 3])
def test_linear_widths(lib, B):
    s, h, _ = lib
    x, y = z(B, 256), z(B, 96)
    s.sffn_linear_forward(h, x, y)
    s.sffn_linear_forward(h, x, y, y)
    s.sffn_linear_forward(h, z(B, 300)[:, :256], z(B, 100)[:, 4:], z(B, 97)[:, :96])     # views with longer rows
    s.sffn_linear_forward(h, x.view(B, 4, 64), y.view(B, 3, 32), y.view(B, 3, 32))        # heads beside each other
    s.sffn_linear_forward(h, z(B, 2, 256)[:, 1:], y)
    assert s.calls == ["sffn_linear_forward"] * 5
    for bad in ((z(B, 255), y), (z(B, 8), y), (z(B, 512), y), (x, z(B, 8)), (x, z(B, 97)), (x, z(B + 1, 96)),
                (x, y, z(B, 8)), (x, y, z(B + 1, 96)), (z(B, 4, 128)[..., :64], y), (x, z(B, 3, 64)[..., :32]),
                (x, y.view(B, 3, 32), z(B, 3, 64)[..., :32]), (z(B, 4, 32), y), (z(B, 1, 4, 64), y)):
        with pytest.raises(ValueError):
            s.sffn_linear_forward(h, *bad)
    assert len(s.calls) == 5


def test_linear_pack_sizes(lib):
    s, h, _ = lib
    codes, scales, bias = z(96, 256, dtype=torch.int8), z(96, 4, dtype=torch.float16), z(96)
    s.sffn_linear_pack(h, codes, scales, None, bias)
    s.sffn_linear_pack(h, codes.data_ptr(), scales.data_ptr())
    assert s.calls == ["sffn_linear_pack"] * 2
    for bad in ((codes[:8], scales), (codes, scales[:, :2]), (codes, scales.float()), (codes.short(), scales),
                (codes, scales, None, bias[:8]), (codes, scales, None, bias.half()), (codes, scales, scales[:1]),
                (z(256, 96, dtype=torch.int8).T, scales)):
        with pytest.raises(ValueError):
            s.sffn_linear_pack(h, *bad)
    assert len(s.calls) == 2


def batch(s, n):
    return s.KvBatch(z(1, 4, dtype=torch.int32), z(1, dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32), n)


@pytest.mark.parametrize("n", [1, 2])
def test_cache_heads_and_widths(lib, n):
    s, _, c = lib
    b, k, q, lse = batch(s, n), z(n, 3, 64), z(n, 6, 64), z(n, 6)
    s.sffn_kv_append(c, b, None, k, k)
    s.sffn_kv_append(c, b, q, k, k, q)
    s.sffn_kv_gather(c, b, k, k)
    s.sffn_kv_gather(c, b, None, k)
    s.sffn_attend(c, b, q, z(n, 6, 64), lse, 1.0)
    assert len(s.calls) == 5
    for bad in ((None, z(n, 2, 64), k), (None, k, z(n, 2, 64)), (None, z(n, 3, 32), z(n, 3, 32)), (None, z(n, 4, 64), k),
                (None, z(n + 1, 3, 64), k), (None, z(n, 192), k), (z(n, 6, 32), k, k, z(n, 6, 32)),
                (z(n, 384), k, k, z(n, 384)), (q, k, k, z(n, 5, 64)), (z(n + 1, 6, 64), k, k, z(n + 1, 6, 64))):
        with pytest.raises(ValueError):
            s.sffn_kv_append(c, b, *bad)
    for bad in ((z(n, 2, 64), k), (k, z(n, 2, 64)), (z(n, 3, 32), None), (None, z(n + 1, 3, 64)), (None, z(n, 192))):
        with pytest.raises(ValueError):
            s.sffn_kv_gather(c, b, *bad)
    for bad in ((z(n, 6, 32), z(n, 6, 32), None), (q, z(n, 5, 64), None), (q, z(n, 6, 32), None), (z(n, 384), z(n, 384), None),
                (z(n + 1, 6, 64), z(n + 1, 6, 64), None), (q, q, z(n, 5))):
        with pytest.raises(ValueError):
            s.sffn_attend(c, b, *bad, 1.0)
    assert len(s.calls) == 5


def test_one_key_head_may_come_without_its_dimension(lib):
    s, _, _ = lib
    s._lib.sffn_kv_get_desc = lambda handle, out: [setattr(out._obj, "n_kv_heads", 1), setattr(out._obj, "head_dim", 64)] and 0
    k = z(2, 64)                                             # and a handle that the binding did not make
    s.sffn_kv_append(77, batch(s, 2), None, k, k)
    s.sffn_kv_gather(77, batch(s, 2), k, k)
    with pytest.raises(ValueError):
        s.sffn_kv_gather(77, batch(s, 2), z(2, 32), None)
    assert len(s.calls) == 2


def test_sizes_go_with_the_handle(lib):
    s, h, c = lib
    assert s._linear_sizes[h] == (256, 96) and s._kv_sizes[c] == (3, 64)
    s.sffn_linear_destroy(h)
    s.sffn_kv_destroy(c)
    assert h not in s._linear_sizes and c not in s._kv_sizes
