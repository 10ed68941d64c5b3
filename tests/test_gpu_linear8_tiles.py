"""8-bit linear layer for many tokens where few tiles are left over after whole waves, and for
few where their codes fill a block's shared memory: bits against a plain implementation."""

import math

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


def layer(sffn, n, k, rows, seed=0):
    """(layer, x, scales of x, its outputs in fp32, bit by bit)."""
    g = gen(seed)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randint(-128, 128, (rows, k), generator=g, device="cuda", dtype=torch.int8)
    scales = (0.5 + torch.rand(n, generator=g, device="cuda")) / (5000 * math.sqrt(k))
    xs, bias = 0.5 + torch.rand(rows, generator=g, device="cuda"), torch.randn(n, generator=g, device="cuda")
    want = R.linear8(x, R.f32(xs), w, R.f32(scales), R.f32(bias), None, "f32").to("cuda")
    return sffn.Linear8.from_weights(w, scales, bias, max_batch=rows), x, xs, want


# (outputs, inputs, tokens): one to three tiles left over, alone or after whole waves (13 x 76 + 1 tiles)
TILES = [(256, 4096, 64), (512, 4096, 100), (128, 8192, 192), (256, 8192, 33), (64, 8192, 100), (700, 2688, 150),
         (256, 65536, 48), (1024, 8192, 64), (11008, 4096, 4300)]


@pytest.mark.parametrize("n,k,rows", TILES)
def test_few_tiles_left_over(sffn, n, k, rows):
    """Four calls on one workspace, and a layer of another shape after them, whose tickets are the same words."""
    L, x, xs, want = layer(sffn, n, k, rows)
    other, x2, xs2, want2 = layer(sffn, 2560, 8192, 64, 1)
    ws = max((L.workspace(rows), other.workspace(64)), key=len)
    y, y2 = torch.empty_like(want), torch.empty_like(want2)
    for _ in range(4):
        y.fill_(7.0)
        sffn.sffn_linear8_forward(L.handle, x, xs, y, None, ws)
        assert torch.equal(y, want)
    for _ in range(2):
        y2.fill_(7.0)
        sffn.sffn_linear8_forward(other.handle, x2, xs2, y2, None, ws)
        assert torch.equal(y2, want2)
    L.check_error()
    other.check_error()


# wide layers whose clusters hold hundreds of rows, for 17 to 32 tokens, which count as 32; 16 of the widest
@pytest.mark.parametrize("n,k,rows", [(8192, 40960, 24), (5200, 36864, 32), (4561, 42496, 17), (8192, 40960, 16),
                                      (2000, 65536, 31), (200, 42560, 32), (2000, 65536, 16)])
def test_few_tokens_of_wide_layers(sffn, n, k, rows):
    L, x, xs, want = layer(sffn, n, k, rows)
    y = torch.full((rows, n), 7.0, device="cuda")
    sffn.sffn_linear8_forward(L.handle, x, xs, y, None, L.workspace(rows))
    L.check_error()
    assert torch.equal(y, want)
    sffn.sffn_linear8_forward(L.handle, x, xs, y, y, L.workspace(rows))            # the residual in y's place
    assert torch.equal(y, want + want)


@pytest.mark.parametrize("pattern", [0, -1, 0x9e3779b900000000 - 2 ** 64, 0x9e3779b900000007 - 2 ** 64])
def test_workspace_of_any_contents(sffn, pattern):
    """A workspace needs no initialisation, whatever a call that gave up, or another operator, has left in it."""
    for n, k, rows in ((1024, 8192, 64), (10240, 2048, 150), (2560, 8192, 64)):
        L, x, xs, want = layer(sffn, n, k, rows, 2)
        ws = L.workspace(rows)
        y = torch.empty_like(want)
        for _ in range(2):
            y.fill_(7.0)
            ws.view(torch.int64).fill_(pattern)
            sffn.sffn_linear8_forward(L.handle, x, xs, y, None, ws)
            assert torch.equal(y, want)
        L.check_error()
