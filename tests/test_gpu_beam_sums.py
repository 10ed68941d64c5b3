"""Sums of exponentials of the choice of continuations where they are hard to keep exact."""

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


def select(sffn, logits, scores, n_out):
    """(scores float64, parents, tokens) as numpy arrays."""
    batch, beams = scores.shape
    H = sffn.Beams(logits.shape[1], beams, n_out, max_batch=batch)
    out = torch.empty(batch, n_out, device="cuda")
    parents, tokens = torch.empty(2, batch, n_out, dtype=torch.int32, device="cuda")
    sffn.sffn_beam_select(H.handle, logits, scores, out, parents, tokens, ws=H.workspace(batch))
    H.check_error()
    return out.double().cpu().numpy(), parents.cpu().numpy(), tokens.cpu().numpy()


# masks that leave whole parts of a row far below every other logit: those parts take their own largest as reference
@pytest.mark.parametrize("mask", [-1e9, torch.finfo(torch.float32).min])
@pytest.mark.parametrize("at", [0.0, 1000.0, -2000.0, 4.0e6])
def test_masked_parts_beside_large_logits(sffn, at, mask):
    """Off by no more than a row without such parts. What rounding log2 e to a float left (1.3e-8 of each logit, 1.3e-5 at
    1000) is put right in the other parts too."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    z = 2.5 * torch.randn(2, 60000, generator=g, device="cuda") + at
    z[0, :40000] = mask
    z[1, 20000:] = mask
    scores = torch.tensor([[-0.5, -0.75]], device="cuda")
    out, parents, tokens = select(sffn, z, scores, 8)
    want, wp, wt = R.select(z.double().cpu().numpy(), scores[0].double().cpu().numpy(), 8)
    np.testing.assert_array_equal(parents[0], wp)
    np.testing.assert_array_equal(tokens[0], wt)
    assert (np.abs(out[0] - want) <= R.LSE_OFF + 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("at", [0.02, -0.05, 0.12, -0.18])
def test_equal_logits_over_a_long_row(sffn, dtype, at):
    """64 rows that a block each takes alone. Equal terms are rounded the same way at every addition, so that one running
    sum of a lane's 2048 was off by 2^-16. Now: 17 roundings of 2^-24, an argument below 8 rounded to 2^-22 (times log 2),
    an exponential good to 2^-22: together below 2^-19."""
    beams, vocab = 64, 1 << 20
    z = torch.full((beams, vocab), at, dtype=R.TORCH[dtype], device="cuda")
    out, parents, tokens = select(sffn, z, torch.full((1, beams), -1.0, device="cuda"), 64)
    want = -1.0 - math.log(vocab)
    assert (parents == 0).all() and (tokens == np.arange(64)).all()
    assert np.abs(out - want).max() <= 2.0 ** -19 + 2.0 ** -24 * abs(want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_logits_far_from_zero(sffn, dtype):
    """The same beyond 2^22, where a part is summed again, its largest logit the reference."""
    beams, vocab = 64, 1 << 20
    z = torch.full((beams, vocab), -1e9, dtype=R.TORCH[dtype], device="cuda")
    z[:, ::3] = z[:, ::3] * 2                                   # nothing beside the others
    out, parents, tokens = select(sffn, z, torch.full((1, beams), -1.0, device="cuda"), 64)
    want = -1.0 - math.log(vocab - len(range(0, vocab, 3)))
    assert (parents == 0).all() and (tokens == [i for i in range(100) if i % 3][:64]).all()
    assert np.abs(out - want).max() <= 2.0 ** -19 + 2.0 ** -24 * abs(want)


@pytest.mark.parametrize("score", [-1e9, -1e30, torch.finfo(torch.float32).min, 1e30])
@pytest.mark.parametrize("vocab,n_out", [(60000, 12), (3000, 64)])
def test_scores_that_swallow_the_logits(sffn, score, vocab, n_out):
    """Of one sequence the largest logits go on, in their order, whatever its score and however many parts its row has."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    z = 1e-3 * torch.randn(6, vocab, generator=g, device="cuda")
    z[0, ::7] = z[0, 5]                                         # ties of logits go to the lowest token
    order = [np.lexsort((np.arange(vocab), -r))[:n_out] for r in z.double().cpu().numpy()]
    alone = torch.full((6, 1), score, device="cuda")
    for batch in (6, 1):
        out, parents, tokens = select(sffn, z[:batch], alone[:batch], n_out)
        assert (parents == 0).all() and (out[np.isfinite(out)] == alone[0].item()).all()
        np.testing.assert_array_equal(tokens, order[:batch])
    out, parents, tokens = select(sffn, z, alone.view(1, 6), n_out)
    if score != -1e9:                                           # whose totals differ by sequence
        assert (parents == 0).all()
        np.testing.assert_array_equal(tokens[0], order[0])


def test_many_candidates_of_one_total(sffn):
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    z = torch.randn(16, 60000, generator=g, device="cuda")
    out, parents, tokens = select(sffn, z, torch.full((1, 16), -1e30, device="cuda"), 32)
    assert (parents == 0).all()
    np.testing.assert_array_equal(tokens[0], np.argsort(-z[0].cpu().numpy(), kind="stable")[:32])


@pytest.mark.parametrize("above", [0.5, 8.0, 255.0, 300.0])
@pytest.mark.parametrize("limit", [-2.0 ** 22, 2.0 ** 22])
def test_logits_around_the_last_whole_reference(sffn, above, limit):
    """One logit on one side of 2^22 in size, all others on the other, 1.5 below it."""
    z = torch.full((2, 5000), limit + above - 1.5, device="cuda")
    z[:, 777] = limit + above
    z[1, 1000:] = limit - 2.0
    out, parents, tokens = select(sffn, z, torch.tensor([[-1.0, -1.5]], device="cuda"), 3)
    want, wp, wt = R.select(z.double().cpu().numpy(), np.array([-1.0, -1.5]), 3)
    np.testing.assert_array_equal(parents[0], wp)
    np.testing.assert_array_equal(tokens[0], wt)
    assert (np.abs(out[0] - want) <= R.LSE_OFF + 2.0 ** -24 * np.abs(want)).all()
