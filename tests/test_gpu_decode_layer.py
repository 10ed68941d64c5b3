"""The example decoder layer: projections, append, attention, output projection
and sparse FFN of one step together, replayed from a CUDA graph."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("args", [
    ["--workload", "opt6.7b_relu_d4096_f16384_fp16", "--heads", "32", "--kv-heads", "32", "--context", "200", "--steps", "3"],
    ["--workload", "falcon40b_relu_d8192_f32768_fp16_batch", "--heads", "128", "--kv-heads", "8", "--context", "70",
     "--steps", "2", "--batch", "9"],
])
def test_example_runs_and_agrees(example, args):
    r = example.main(args)
    # fp32 on both sides, sums in other orders: each of the two projections off by at most (40 + K / 128) 2^-24 = 6e-6 of its
    # absolute terms, which exceed its result by less than two, and the attention by less
    assert r["finite"] and r["off"] < 2e-5
