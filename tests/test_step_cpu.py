"""Refusals of what stands around the halves of a decode step, without a GPU:
host-side checks of the C calls, and the binding's comparison of tensors with
the sizes of their handle (the library replaced by one that counts calls)."""

import ctypes
import types

import numpy as np
import pytest
import torch

import step_ref as R


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from activation_sparse_ffn_gb300 import sffn
    return sffn


@pytest.mark.parametrize("kw,ok", [
    (dict(in_features=16, out_features=1), True), (dict(in_features=65536, out_features=1 << 20, max_batch=65536), True),
    (dict(in_features=8, out_features=8), False), (dict(in_features=0, out_features=8), False),
    (dict(in_features=4100, out_features=8), False), (dict(in_features=65552, out_features=8), False),
    (dict(in_features=64, out_features=0), False), (dict(in_features=64, out_features=(1 << 20) + 1), False),
    (dict(in_features=64, out_features=8, max_batch=0), False), (dict(in_features=64, out_features=8, max_batch=65537), False)])
def test_linear8_validate(lib, kw, ok):
    assert lib.sffn_linear8_validate(lib.make_linear8_desc(**kw)) == (0 if ok else lib.SFFN_ERR_INVALID_ARG)


@pytest.mark.parametrize("kw,ok", [
    (dict(vocab=1, beams=1, n_out=1), True), (dict(vocab=1 << 24, beams=64, n_out=64, max_batch=1023), True),
    (dict(vocab=0, beams=1, n_out=1), False), (dict(vocab=(1 << 24) + 1, beams=1, n_out=1), False),
    (dict(vocab=5, beams=0, n_out=1), False), (dict(vocab=5, beams=65, n_out=1), False),
    (dict(vocab=5, beams=1, n_out=0), False), (dict(vocab=5, beams=1, n_out=65), False),
    (dict(vocab=5, beams=1, n_out=1, max_batch=0), False), (dict(vocab=5, beams=64, n_out=1, max_batch=1024), False)])
def test_beam_validate(lib, kw, ok):
    assert lib.sffn_beam_validate(lib.make_beam_desc(**kw)) == (0 if ok else lib.SFFN_ERR_INVALID_ARG)


def test_host_refusals(lib):
    L, bad, Rows = lib._lib, lib.SFFN_ERR_INVALID_ARG, lib.RowsC
    r, none = Rows(4096, 64, 0), Rows()

    def norm(x=r, res=none, w=None, eps=1e-5, n=2, width=64, s=none, y=r, q=none, sc=None, t=0, yt=0):
        return L.sffn_norm(x, res, w, eps, n, width, s, y, q, sc, t, yt, None)

    y = Rows(8192, 64, 0)
    for kw in (dict(n=-1), dict(n=(1 << 30) + 1), dict(width=0), dict(width=32769), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(t=3), dict(yt=-1), dict(y=none), dict(x=none), dict(x=Rows(4097, 64, 0)),
               dict(x=Rows(4096, 63, 0)), dict(res=Rows(4098, 64, 0)), dict(s=Rows(16384, 60, 0)), dict(w=4097),
               dict(y=y, s=y), dict(y=r, yt=1), dict(y=r, t=2, yt=0, x=r), dict(y=none, q=y), dict(y=none, q=y, sc=6),
               dict(y=none, q=Rows(8192, 63, 0), sc=4)):
        assert norm(**kw) == bad, kw
    assert norm(n=0) == 0
    assert L.sffn_quantize(none, 0, 64, none, None, 0, None) == 0
    for args in ((r, -1, 64, y, 4096, 0), (r, 1, 0, y, 4096, 0), (r, 1, 65537, y, 4096, 0), (r, 1, 64, y, 4096, 5),
                 (none, 1, 64, y, 4096, 0), (r, 1, 64, none, 4096, 0), (r, 1, 64, y, None, 0), (r, 1, 64, y, 4098, 0)):
        assert L.sffn_quantize(*args, None) == bad, args
    out = ctypes.c_void_p()
    for create in (L.sffn_linear8_create, L.sffn_beam_create):
        assert create(None, ctypes.byref(out)) == bad and create(None, None) == bad and out.value is None
    assert L.sffn_linear8_pack(None, None, None, None, None) == bad
    assert L.sffn_linear8_forward(None, r, None, 1, none, y, 0, None, 0, None) == bad
    assert L.sffn_linear8_workspace_bytes(None, 1) == 0 and L.sffn_beam_workspace_bytes(None, 1) == 0
    assert L.sffn_linear8_check_error(None, None) == bad and L.sffn_beam_check_error(None, None) == bad
    assert L.sffn_linear8_get_desc(None, None) == bad and L.sffn_beam_get_desc(None, None) == bad
    assert L.sffn_beam_select(None, r, None, None, 0, 1, None, None, None, 0, None, 0, None) == bad
    assert L.sffn_kv_reorder(None, 1, None, None, 1, None, 1, None) == bad
    assert L.sffn_kv_reorder((ctypes.c_void_p * 1)(None), 1, None, None, 1, None, 1, None) == bad
    assert L.sffn_kv_reorder((ctypes.c_void_p * 1)(None), 129, None, None, 1, None, 1, None) == bad
    L.sffn_linear8_destroy(None)
    L.sffn_beam_destroy(None)


@pytest.fixture()
def fake(lib, monkeypatch):
    calls = []

    def take(name):
        def f(*args):
            calls.append(name)
            return 0
        return f

    def create(handle):
        def f(desc, out):
            out._obj.value = handle
            return 0
        return f

    def get_desc(made):
        def f(handle, out):
            for n, _ in out._obj._fields_:
                setattr(out._obj, n, getattr(made, n))
            return 0
        return f

    linear, beam = lib.make_linear8_desc(256, 96, 8), lib.make_beam_desc(50, 3, 6, 4)
    monkeypatch.setattr(lib, "_lib", types.SimpleNamespace(
        sffn_linear8_create=create(4096), sffn_beam_create=create(8192),
        sffn_linear8_get_desc=get_desc(linear), sffn_beam_get_desc=get_desc(beam),
        **{n: take(n) for n in ("sffn_norm", "sffn_quantize", "sffn_linear8_pack", "sffn_linear8_forward",
                                "sffn_linear8_destroy", "sffn_beam_select", "sffn_beam_destroy", "sffn_kv_reorder")}))
    monkeypatch.setattr(lib, "_stream", lambda stream: None)
    h, b = lib.sffn_linear8_create(linear), lib.sffn_beam_create(beam)
    yield lib, h, b, calls
    lib.sffn_linear8_destroy(h)
    lib.sffn_beam_destroy(b)


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


I8, I32 = torch.int8, torch.int32


def test_norm_sizes(fake):
    s, _, _, calls = fake
    x, w = z(3, 64), z(64)
    s.sffn_norm(x, w, 1e-5, x, x, z(3, 64, dtype=torch.bfloat16))
    s.sffn_norm(x.view(3, 4, 16), None, 1e-5, y=x)
    s.sffn_norm(x, codes=z(3, 64, dtype=I8), scales=z(3))
    s.sffn_quantize(z(3, 2, 32), z(3, 64, dtype=I8), z(3))
    assert len(calls) == 4
    for kw in (dict(weight=z(63)), dict(weight=z(64).half()), dict(residual=z(3, 65)), dict(residual=z(2, 64)),
               dict(residual=z(3, 64).half()), dict(sum=z(3, 64).half()), dict(sum=z(4, 64)), dict(y=z(3, 32)),
               dict(y=z(3, 64, dtype=torch.float64)), dict(codes=z(3, 64, dtype=I8)), dict(codes=z(3, 64), scales=z(3)),
               dict(codes=z(3, 64, dtype=I8), scales=z(2)), dict(codes=z(3, 64, dtype=I8), scales=z(3).half()),
               dict(y=z(64, 3).t())):
        with pytest.raises(ValueError):
            s.sffn_norm(x, **kw)
    for bad in ((z(64), z(1, 64, dtype=I8), z(1)), (x, z(3, 60, dtype=I8), z(3)), (x, z(3, 64), z(3)),
                (x, z(3, 64, dtype=I8), z(4)), (z(3, 4, 32)[..., :16], z(3, 64, dtype=I8), z(3))):
        with pytest.raises(ValueError):
            s.sffn_quantize(*bad)
    assert len(calls) == 4


def test_linear8_sizes(fake):
    s, h, _, calls = fake
    x, xs, y = z(5, 256, dtype=I8), z(5), z(5, 96)
    s.sffn_linear8_forward(h, x, xs, y)
    s.sffn_linear8_forward(h, x, xs, y, y)
    s.sffn_linear8_forward(h, z(5, 272, dtype=I8)[:, 16:], xs, z(5, 100)[:, 4:])
    s.sffn_linear8_forward(h, x, xs, z(5, 3, 32))
    s.sffn_linear8_pack(h, z(96, 256, dtype=I8), z(96), z(96))
    assert len(calls) == 5
    for bad in ((z(5, 255, dtype=I8), xs, y), (z(5, 256), xs, y), (x, z(4), y), (x, z(5).half(), y), (x, xs, z(4, 96)),
                (x, xs, z(5, 97)), (x, xs, y, z(5, 96).half()), (x, xs, y, z(5, 95)), (x, xs, y.double())):
        with pytest.raises(ValueError):
            s.sffn_linear8_forward(h, *bad)
    for bad in ((z(96, 255, dtype=I8), z(96)), (z(96, 256), z(96)), (z(96, 256, dtype=I8), z(95)),
                (z(96, 256, dtype=I8), z(96).half()), (z(96, 256, dtype=I8), z(96), z(97))):
        with pytest.raises(ValueError):
            s.sffn_linear8_pack(h, *bad)
    assert len(calls) == 5


def test_beam_sizes(fake):
    s, _, b, calls = fake
    logits, scores, out = z(6, 50), z(2, 3), (z(2, 6), z(2, 6, dtype=I32), z(2, 6, dtype=I32))
    s.sffn_beam_select(b, logits, scores, *out)
    s.sffn_beam_select(b, logits.half(), scores, *out, z(2, 3, dtype=torch.bool), 4)
    assert len(calls) == 2
    for bad in ((z(5, 50), scores, *out), (z(6, 49), scores, *out), (logits, z(2, 2), *out), (logits, scores.half(), *out),
                (logits, scores, z(2, 5), *out[1:]), (logits, scores, out[0], z(2, 6), out[2]),
                (logits, scores, *out[:2], z(2, 6, dtype=torch.int64)), (logits, scores, *out, z(2, 3)),
                (logits, scores, *out, z(3, dtype=torch.uint8)), (logits.double(), scores, *out)):
        with pytest.raises(ValueError):
            s.sffn_beam_select(b, *bad)
    assert len(calls) == 2


def test_reference_of_continuations_against_brute_force():
    """select() against the definition written out: every total, sorted by (total, place)."""
    rng = np.random.default_rng(0)
    logits, scores = rng.integers(0, 4, (3, 9)).astype(np.float64), np.array([-1.0, -1.0, -3.0])
    logits[1, 2:5] = -np.inf
    every = []
    for j in range(3):
        lse = np.log(np.exp(logits[j]).sum())
        every += [(-(scores[j] + v - lse), j, t) for t, v in enumerate(logits[j]) if v > -np.inf]
    got = R.select(logits, scores, 7)
    want = sorted((round(v, 12), j, t) for v, j, t in every)[:7]
    assert [(j, t) for _, j, t in want] == list(zip(got[1].tolist(), got[2].tolist()))
    assert np.allclose(got[0], [-v for v, _, _ in want])
    assert R.select(np.full((2, 4), -np.inf), np.zeros(2), 3)[0].tolist() == [-np.inf] * 3


def test_reference_of_codes():
    y = np.array([[127.0, 0.5, 1.5, -2.5, -127.0], [0, 0, 0, 0, 0], [1, np.nan, 0, 0, 0], [np.inf, 1, 0, 0, 0]], np.float32)
    q, s = R.codes(y)
    assert q.tolist() == [[127, 0, 2, -2, -127], [0] * 5, [0] * 5, [0] * 5]
    assert s[0] == 1 and s[1] == 0 and np.isnan(s[2:]).all()
