"""Norm of more rows than blocks: each block takes several, one warp or many."""

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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [8, 104, 256, 264, 2048])
def test_norm_of_many_short_rows(sffn, dtype, width):
    """Rows of very different sizes beside each other, so that a factor or a largest element of another row shows."""
    rows = 6000
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    size = torch.exp2(torch.randint(-12, 13, (rows, 1), generator=g, device="cuda").float())
    x = (size * torch.randn(rows, width, generator=g, device="cuda")).to(R.TORCH[dtype])
    w = 1 + 0.2 * torch.randn(width, generator=g, device="cuda")
    y = torch.empty_like(x)
    codes, scales = torch.empty(rows, width, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    sffn.sffn_norm(x, w, 1e-5, None, None, y, codes, scales)
    _, want = R.norm(R.f32(x), None, R.f32(w), 1e-5)
    q, s = R.codes(want)
    assert torch.equal(y.cpu(), R.rounded(want, dtype))
    assert torch.equal(scales.cpu(), torch.from_numpy(s))
    assert torch.equal(codes.cpu(), torch.from_numpy(q))
