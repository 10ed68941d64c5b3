"""The operators around the halves together, as a beam search uses them
(examples/beam_search.py): eager and replayed from a CUDA graph, against the
score of the same sequence fed alone, and on streams of their own."""

import os
import sys
import threading

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    import beam_search
    return beam_search


def test_graph_replays_the_eager_search(example):
    """The same bits: a cache that beams share, pages that end on the way (24 steps, pages of 16)."""
    d = example.Decoder(batch=3, beams=4, ffn=False)
    eager, graph = d.run(24, graph=False), d.run(24)
    assert torch.equal(eager[0], graph[0]) and torch.equal(eager[1], graph[1])
    assert bool((eager[1][:, :-1] >= eager[1][:, 1:]).all())


def test_scores_are_those_of_the_sequences_alone(example):
    """A beam's score against that of its tokens fed to one row with a cache of its own. Sums of 8-bit codes and norms do
    not depend on the batch; attention's order of sums does, by 2^-20 of its result, which moves a code of its 8-bit rows
    by one in at most 2^-20 * 127 * 2 of the elements, and a logit by then at most 1/127 of a unit times that
    element's share: below 1e-3 a step in all."""
    d, alone = example.Decoder(batch=2, beams=4, ffn=False), example.Decoder(batch=1, beams=1, ffn=False)
    sequences, scores = d.run(20)
    for b in range(2):
        for j in (0, 3):
            assert abs(alone.score_of(sequences[b, j].tolist()) - float(scores[b, j])) < 20 * 1e-3
    assert len({tuple(s) for s in sequences[0].tolist()}) == 4      # four different sequences


def test_example_runs(example, capsys):
    out = example.main(["--steps", "18"])
    assert "us per step" in capsys.readouterr().out
    assert bool(out["scores"].isfinite().all()) and out["sequences"].shape == (2, 4, 18)


def test_two_searches_at_once(example):
    """From two threads, on a stream each, with weights of their own."""
    made = [example.Decoder(batch=2, beams=4, ffn=False, seed=s) for s in (0, 1)]
    want = [d.run(12, graph=False) for d in made]
    got = [None, None]

    def go(i):
        got[i] = made[i].run(12, graph=False)

    threads = [threading.Thread(target=go, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("rows", [3, 50, 200])
def test_one_layer_on_two_streams(example, rows):
    """Two calls of one 8-bit layer at once, a workspace each; contents of the workspaces do not matter."""
    from activation_sparse_ffn_gb300 import sffn
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    layer = example.random_linear8(3000, 2048, rows, g)
    x = torch.randint(-127, 128, (2, rows, 2048), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand(2, rows, generator=g, device="cuda")
    y, ws = torch.empty(2, 6, rows, 3000, device="cuda"), [layer.workspace(rows) for _ in range(2)]
    for w in ws:
        w.copy_(torch.randint(0, 256, w.shape, generator=g, device="cuda", dtype=torch.uint8))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(6):
        for i, st in enumerate(streams):
            sffn.sffn_linear8_forward(layer.handle, x[i], s[i], y[i, k], None, ws[i], stream=st)
    torch.cuda.synchronize()
    layer.check_error()
    for i in range(2):
        want = torch.empty(rows, 3000, device="cuda")
        sffn.sffn_linear8_forward(layer.handle, x[i], s[i], want, None, ws[i])
        assert all(torch.equal(y[i, k], want) for k in range(6))


def test_graphs_that_share_a_workspace(example):
    """Two captured selections of one handle and workspace, replayed in turn."""
    from activation_sparse_ffn_gb300 import sffn
    H = sffn.Beams(20000, 4, 8, max_batch=2)
    ws = H.workspace(2)
    z = [torch.randn(8, 20000, device="cuda"), torch.randn(8, 20000, device="cuda")]
    scores = torch.zeros(2, 4, device="cuda")
    out = [(torch.empty(2, 8, device="cuda"), *torch.empty(2, 2, 8, dtype=torch.int32, device="cuda")) for _ in z]
    graphs, stream = [], torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for a, o in zip(z, out):
            sffn.sffn_beam_select(H.handle, a, scores, *o, ws=ws)
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                sffn.sffn_beam_select(H.handle, a, scores, *o, ws=ws)
        stream.synchronize()
        want = [[t.clone() for t in o] for o in out]
        for _ in range(5):
            for g, o in zip(graphs, out):
                for t in o:
                    t.zero_()
                g.replay()
        stream.synchronize()
    assert all(torch.equal(a, b) for w, o in zip(want, out) for a, b in zip(w, o))
    H.check_error()
