"""Element types through paths of the attention half that the other GPU tests
reach with one type only: fp16 rows of projections in every batch size and over
long rows, non-finite numbers and wide ranges with few and with many columns,
NaN slots and non-finite queries of 16-bit rows."""

import pytest
import torch

import attn_ref as R
from test_gpu_attention import TORCH, Case, check_attention, check_linear, gen, host, poison, sffn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [1, 2, 5, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("k,group", [(96, 32), (4096, 128), (11008, 32), (65536, 64)])
def test_linear_fp16_rows(sffn, B, k, group):
    """One run of inputs to several batches of runs a warp, with and without zeros."""
    check_linear(sffn, 70, k, group, B, "f16", zeros=B % 2 == 0, bias=True, residual=B % 3 == 0, seed=B)


@pytest.mark.parametrize("B", [1, 3, 7])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_long_rows_of_few_tokens(sffn, B, dtype):
    check_linear(sffn, 70, 65536, 32, B, dtype, zeros=True, seed=B)


@pytest.mark.parametrize("dtype,B", [("f32", 2), ("f32", 4), ("f32", 9), ("bf16", 5), ("bf16", 8), ("bf16", 20)])
def test_linear_range_of_inputs(sffn, dtype, B):
    """Tokens of very small and very large numbers, a zero token, a wide spread and one huge element."""
    x = torch.randn(B, 1024, generator=gen(3), device="cuda")
    for b in range(B):
        kind = b % 5 if B > 2 else 3 + b
        if kind == 0:
            x[b] *= 1e-30
        elif kind == 1:
            x[b] *= 1e30
        elif kind == 2:
            x[b] = 0
        elif kind == 3:
            x[b, 17] = 1e6
        else:
            x[b] *= torch.logspace(-9, 3, 1024, device="cuda")
    check_linear(sffn, 64, 1024, 128, B, dtype, x=x.to(TORCH[dtype]), seed=9)


@pytest.mark.parametrize("dtype,B", [("f32", 3), ("f16", 3), ("bf16", 5), ("f16", 12), ("bf16", 30)])
@pytest.mark.parametrize("zeros", [False, True])
def test_linear_non_finite_tokens_stay_apart(sffn, dtype, B, zeros):
    lin, x, y, _ = check_linear(sffn, 130, 512, 64, B, dtype, zeros=zeros, seed=4)
    x = x.clone()
    x[1, 100] = float("nan")
    x[2, 5] = float("inf")
    z = torch.empty_like(y)
    sffn.sffn_linear_forward(lin.handle, x, z, None, lin.workspace(B))
    rest = [b for b in range(B) if b not in (1, 2)]
    assert not z[[1, 2]].isfinite().any()
    assert torch.equal(z[rest], y[rest])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("P", [16, 64])
def test_attention_of_16_bit_rows_never_uses_what_it_does_not_see(sffn, dtype, P):
    lens = [(65, 2), (1, 1), (31, 3), (130, 1)]
    for D, G in ((128, 32), (64, 64)):
        c = Case(sffn, lens, 2, D, G, P, dtype, seed=18)
        poison(sffn, c)
        c.fill_cache(sffn)
        check_attention(sffn, lens, 8, 2, D, G, P, dtype, case=c)
        check_attention(sffn, lens, 8, 2, D, G, P, dtype, case=c, window=20)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_non_finite_query_rows_of_16_bits_stay_apart(sffn, dtype):
    c, q, out, lse = check_attention(sffn, [(100, 3)], 8, 2, 64, 64, 16, dtype, seed=19)
    q2 = q.clone()
    q2[1, 3, 5] = float("nan")
    q2[2, 6, 0] = float("inf")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    sffn.sffn_attend(c.cache.handle, c.new, q2, o2, l2, 1 / 8, 0, c.cache.workspace(c.new, 8))
    bad = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[2, 6] = True
    assert o2[bad].isnan().all()
    assert torch.equal(o2[~bad], out[~bad]) and torch.equal(l2[~bad], lse[~bad])


def test_append_extreme_rows_of_16_bits(sffn):
    for dtype in ("f16", "bf16"):
        c = Case(sffn, [(8, 8)], 1, 128, 64, 16, dtype, seed=2)
        k = c.randn(8, 1, 128)
        k[0] = 3.25
        k[1] = 0
        k[2] *= 1e-6
        k[3] *= 1e4
        k[4, 0, 3] = float("inf")
        k[5, 0, 100] = float("nan")
        k[6] = -6e4
        k[7, 0, :64] = 6e-8
        sffn.sffn_kv_append(c.cache.handle, c.new, None, k, k)
        want = R.stored(k.float().cpu().numpy(), 64)
        ko, vo = torch.empty(8, 1, 128, device="cuda"), torch.empty(8, 1, 128, device="cuda")
        sffn.sffn_kv_gather(c.cache.handle, c.new, ko, vo)
        for got in (ko, vo):
            assert torch.equal(got.cpu().nan_to_num(7.0), torch.from_numpy(want).nan_to_num(7.0))
        c.cache.check_error()
