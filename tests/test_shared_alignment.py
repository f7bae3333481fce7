"""Kernels that access their dynamic shared memory as vectors declare it aligned to them: without that its place
follows from the sizes of the static arrays in front of it."""

import os
import re

import pytest

from bwd_flashattention_fwd_sm_gb300.build import CSRC

DECLARED = re.compile(r"extern __shared__ (?:__align__\((\d+)\) )?([\w ]+?) (\w+)\[\];")


@pytest.mark.parametrize("name", ["embed.cu", "ln.cu", "ln_bwd.cuh", "ln_drop.cuh"])
def test_row_operators_declare_the_alignment_of_their_vectors(name):
    with open(os.path.join(CSRC, name)) as f:
        source = f.read()
    found = DECLARED.findall(source)
    assert found and len(found) == source.count("extern __shared__")
    for align, kind, array in found:
        # float arrays are accessed by elements, everything else as 16-byte vectors, pairs of words or bulk copies
        assert kind == "float" or int(align or 0) >= 16, (name, kind, array)
