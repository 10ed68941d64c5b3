"""The attention half of a decode step without a GPU: host-side checks of
descriptions and arguments, sizes, and the plain implementations the GPU tests
compare against."""

import ctypes

import numpy as np
import pytest
import torch

import attn_ref as R


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from activation_sparse_ffn_gb300 import sffn
    return sffn


@pytest.mark.parametrize("kw,ok", [
    (dict(in_features=8192, out_features=10240, group=128, scale_dtype="f16"), True),
    (dict(in_features=32, out_features=1, group=32, scale_dtype="bf16", has_zero=True, max_batch=32), True),
    (dict(in_features=96, out_features=3, group=32, scale_dtype="f32"), True),
    (dict(in_features=65536, out_features=1 << 20, group=64, scale_dtype="f32"), True),
    (dict(in_features=96, out_features=3, group=64, scale_dtype="f32"), False),        # not a multiple of group
    (dict(in_features=96, out_features=3, group=48, scale_dtype="f32"), False),
    (dict(in_features=0, out_features=3, group=32, scale_dtype="f32"), False),
    (dict(in_features=65536 + 32, out_features=3, group=32, scale_dtype="f32"), False),
    (dict(in_features=32, out_features=0, group=32, scale_dtype="f32"), False),
    (dict(in_features=32, out_features=(1 << 20) + 1, group=32, scale_dtype="f32"), False),
    (dict(in_features=32, out_features=8, group=32, scale_dtype=3), False),
    (dict(in_features=32, out_features=8, group=32, scale_dtype="f16", max_batch=0), False),
    (dict(in_features=32, out_features=8, group=32, scale_dtype="f16", max_batch=33), False),
])
def test_linear_validate(lib, kw, ok):
    rc = lib.sffn_linear_validate(lib.make_linear_desc(**kw))
    assert rc == (lib.SFFN_OK if ok else lib.SFFN_ERR_INVALID_ARG), lib.last_error()


@pytest.mark.parametrize("args,ok", [
    ((1, 16, 1, 64, 32), True), ((5, 32, 8, 128, 128), True), ((2 ** 31 - 1, 64, 1024, 256, 64), True),
    ((0, 16, 1, 64, 32), False), ((1, 8, 1, 64, 32), False), ((1, 128, 1, 64, 32), False),
    ((1, 16, 0, 64, 32), False), ((1, 16, 1025, 64, 32), False), ((1, 16, 1, 96, 32), False),
    ((1, 16, 1, 64, 128), False), ((1, 16, 1, 128, 16), False),
])
def test_kv_validate_and_bytes(lib, args, ok):
    desc = lib.make_kv_desc(*args)
    assert lib.sffn_kv_validate(desc) == (lib.SFFN_OK if ok else lib.SFFN_ERR_INVALID_ARG), lib.last_error()
    n, P, H, D, G = args
    assert lib.sffn_kv_bytes(desc) == (n * P * H * (D + 8 * (D // G)) if ok else 0)


def test_null_arguments_are_rejected_on_the_host(lib):
    L, rows, out = lib._lib, lib.RowsC(), ctypes.c_void_p()
    bad = lib.SFFN_ERR_INVALID_ARG
    batch = lib.KvBatchC()
    assert L.sffn_linear_validate(None) == bad and L.sffn_kv_validate(None) == bad
    assert L.sffn_linear_create(None, ctypes.byref(out)) == bad and L.sffn_kv_create(None, ctypes.byref(out)) == bad
    assert L.sffn_linear_create(ctypes.byref(lib.make_linear_desc(32, 1, 32, "f16")), None) == bad
    assert L.sffn_linear_pack(None, None, None, None, None, None) == bad
    assert L.sffn_linear_forward(None, rows, 1, rows, rows, 0, None, 0, None) == bad
    assert L.sffn_linear_get_desc(None, None) == bad and L.sffn_kv_get_desc(None, None) == bad
    assert L.sffn_linear_workspace_bytes(None, 1) == 0
    assert L.sffn_kv_append(None, ctypes.byref(batch), rows, 0, rows, rows, rows, None, 0, None) == bad
    assert L.sffn_kv_gather(None, ctypes.byref(batch), rows, rows, 0, None) == bad
    assert L.sffn_attend(None, ctypes.byref(batch), rows, 1, rows, None, 1.0, 0, 0, None, 0, None) == bad
    assert L.sffn_attend_workspace_bytes(None, 1, 1, 1) == 0
    assert L.sffn_kv_check_error(None, None) == bad and L.sffn_linear_check_error(None, None) == bad
    assert L.sffn_kv_bytes(None) == 0
    assert "NULL" in lib.last_error()
    L.sffn_linear_destroy(None)
    L.sffn_kv_destroy(None)
    assert out.value is None


def test_binding_refuses_mismatched_tensors(lib):
    t = torch.zeros(4, 3, 64)
    with pytest.raises(ValueError):
        lib._rows(t.transpose(1, 2))
    with pytest.raises(ValueError):
        lib._rows(torch.zeros(4))
    with pytest.raises(ValueError):
        lib._rows(t, torch.float16, "x")
    with pytest.raises(ValueError):
        lib._io_dtype(torch.float64)
    r = lib._rows(t[:, 1:])
    assert (r.row_stride, r.head_stride, r.ptr) == (192, 64, t.data_ptr() + 256)
    with pytest.raises(ValueError):
        lib.KvBatch(torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    b = lib.KvBatch(torch.zeros(2, 4, dtype=torch.int32)[:, :3], torch.zeros(2, dtype=torch.int32))
    assert (b.c.table_stride, b.c.n_seq, b.c.n_tokens) == (4, 2, 2)


# ------------------------------------------------------------------ the plain implementations

def test_stored_rows_by_hand():
    # 0 .. 15 in one group: mid 7.5, step 0.5, every value is a level
    x = np.zeros((1, 32), np.float32)
    x[0, :16] = np.arange(16)
    x[0, 16:] = 7.6
    want = x.copy()
    want[0, 16:] = 8
    assert np.array_equal(R.stored(x, 32), want)
    # a constant group is held exactly if it is a half-precision number; ties go up
    assert np.array_equal(R.stored(np.full((1, 32), -2.5, np.float32), 32), np.full((1, 32), -2.5))
    y = np.zeros((1, 32), np.float32)
    y[0, 0], y[0, 1] = 15, 1.5
    assert R.stored(y, 32)[0, 1] == 2
    # the error is at most one step (half a level), and the half-precision rounding of mid and step
    z = np.random.default_rng(0).standard_normal((50, 128)).astype(np.float32)
    step, _, _ = R.group_params(z, 64)
    off = np.abs(R.stored(z, 64) - z).reshape(50, 2, 64).max(-1)
    assert (off <= step.astype(np.float32) * (1 + 2.0 ** -6)).all()
    bad = z.copy()
    bad[3, 70] = np.inf
    held = R.stored(bad, 64)
    assert np.isnan(held[3, 64:]).all() and np.isfinite(np.delete(held, 3, 0)).all() and np.isfinite(held[3, :64]).all()


def test_rotation_by_hand():
    x = np.arange(8, dtype=np.float32).reshape(1, 1, 8)
    quarter = np.array([[[0, 1], [1, 0]]], np.float32)              # pair 0 a quarter turn, pair 1 none
    assert R.rotate(x, quarter, "halves").ravel().tolist() == [-2, 1, 0, 3, 4, 5, 6, 7]
    assert R.rotate(x, quarter, "pairs").ravel().tolist() == [-1, 0, 2, 3, 4, 5, 6, 7]


def test_attention_by_hand():
    k = np.array([[[1.0, 0]], [[0, 1.0]], [[1.0, 1.0]]])
    v = np.array([[[1.0, 2]], [[3, 4]], [[5, 6]]])
    q = np.zeros((4, 2, 2))
    out, lse, _ = R.attention(q, k, v, 4, 1.0, 0)                   # four rows, three positions: the first sees none
    assert np.array_equal(out[0], np.zeros((2, 2))) and np.isneginf(lse[0]).all()
    assert np.allclose(out[1], [1, 2]) and np.allclose(out[3], [3, 4]) and np.allclose(lse[3], np.log(3))
    out, lse, _ = R.attention(q, k, v, 4, 1.0, 1)
    assert np.allclose(out[3], [5, 6]) and np.allclose(lse[3], 0)


def test_linear_by_hand():
    x, codes = np.array([[1.0, 2, 3, 4]]), np.array([[1, -1, 7, -8]])
    y, _ = R.linear(x, codes, np.array([[0.5, 2]]), np.array([[1, 0]]), np.array([10.0]), np.array([[100.0]]), 2)
    assert y[0, 0] == 0.5 * (0 * 1 - 2 * 2) + 2 * (21 - 32) + 110
