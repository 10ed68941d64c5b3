"""What can be told of shared memory from the kernels' sources: dynamic shared memory follows the static arrays of a kernel
with the alignment that its declaration asks for, and kernels read it 16 bytes at a time."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "activation_sparse_ffn_gb300", "csrc")


def declarations():
    """(file, what is declared, the statement after it) of all dynamic shared memory."""
    for file in sorted(os.listdir(CSRC)):
        if file.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, file)) as f:
                for m in re.finditer(r"extern __shared__ ([^;]*);\s*([^;]*);", f.read()):
                    yield file, m[1], m[2]


def test_dynamic_shared_memory_is_aligned_for_its_reads():
    assert len(list(declarations())) >= 10
    for file, what, then in declarations():
        asked = re.search(r"__align__\((\d+)\)", what)
        by_hand = re.search(r"& 1023|~\(?uintptr_t\)?|\+ 1023", then)
        assert (asked and int(asked[1]) % 16 == 0) or what.startswith("uint4 ") or by_hand, f"{file}: {what}"
