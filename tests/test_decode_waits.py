"""Kernels that may be brought in while the one in front of them ends read memory only
behind griddepcontrol.wait, whoever wrote it (read from the sources: nothing promises
the order that another place would rest on, and nothing measurable shows it)."""
import os
import re

import pytest

import hadamard_rotated_activation_b200 as kq

CSRC = os.path.join(os.path.dirname(os.path.abspath(kq.__file__)), "csrc")
READS = re.compile(r"\b(parts_of|join_signs|sequence|begin|look|load_x|stage_x|scan32|sum_parts|fetch|"
                   r"place|__ldg|__ldcg|reinterpret_cast<const|P\.seq_lens|P\.block_table)\b|ld\.global|"
                   r"\*P\.|P\.\w+\[")


@pytest.mark.parametrize("name,kernels", [("kq_attn.cu", 3), ("kq_gemv.cu", 1), ("kq_kvcopy.cu", 1)])
def test_kernels_wait_before_they_read(name, kernels):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    bodies = re.split(r"__global__", text)[1:]
    assert len(bodies) == kernels
    for body in bodies:
        ahead, wait, _ = body.partition('"griddepcontrol.wait;"')
        assert wait
        assert not READS.search(ahead[ahead.index("{"):]), ahead
