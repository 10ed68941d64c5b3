"""What can be told from the kernels' sources: shared-memory barriers are
initialised by some threads of a block and used by others, so that a barrier of
the block that every thread meets has to stand between."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "activation_sparse_ffn_gb300", "csrc")
USES = r"\b(?:mbar_arrive\w*|mbar_wait\w*|mbar_try_wait|bulk_g2s)\s*\("
BARRIERS = r"\b(?:__syncthreads|cluster_barrier)\s*\(\s*\)"


def kernels():
    """(file, name, body) of every kernel that initialises a shared-memory barrier."""
    for file in sorted(os.listdir(CSRC)):
        if not file.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(CSRC, file)) as f:
            text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
        for at in (m.end() for m in re.finditer(r"\b__global__\b", text)):
            begin = text.find("{", at)
            if 0 <= text.find(";", at) < begin:
                continue                                     # a declaration
            depth, end = 1, begin + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            if "mbar_init(" in text[begin:end]:
                yield file, re.findall(r"(\w+)\s*\(", text[at:begin])[-1], text[begin:end]


def unguarded(body):
    """The first use of a barrier that no block barrier separates from the last initialisation, or None. A block barrier
    within braces that were opened after the initialisation does not count: not every thread need meet it."""
    at = body.rindex("mbar_init(")
    low = depth = body[:at].count("{") - body[:at].count("}")
    for m in re.finditer(r"[{}]|" + USES + "|" + BARRIERS, body[at:]):
        if m[0] == "{":
            depth += 1
        elif m[0] == "}":
            depth -= 1
            low = min(low, depth)
        elif re.match(BARRIERS, m[0]):
            if depth == low:
                return None
        else:
            return m[0]
    return None


@pytest.mark.parametrize("file,name,body", [pytest.param(*k, id=f"{k[0]}:{k[1]}") for k in kernels()])
def test_barriers_are_initialised_before_they_are_used(file, name, body):
    assert unguarded(body) is None, f"{file}: {name} reaches {unguarded(body)} without a block barrier after mbar_init"


def test_the_check_sees_what_it_looks_for():
    assert unguarded("{ mbar_init(b); mbar_arrive(b); }") == "mbar_arrive("
    assert unguarded("{ if (t == 0) { mbar_init(b); } __syncthreads(); mbar_arrive(b); }") is None
    assert unguarded("{ mbar_init(b); if (many) { __syncthreads(); } mbar_arrive(b); }") == "mbar_arrive("
    assert unguarded("{ for (;;) { if (first) mbar_init(b); __syncthreads(); bulk_g2s(b); } }") is None
    assert len(list(kernels())) >= 6
