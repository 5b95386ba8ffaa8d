"""A kernel launched with programmatic stream serialization lives from before
its wait on, while the kernel ahead of it still writes.  Non-coherent loads
(__ldg, or a const __restrict__ pointer, which lets the compiler choose them)
are only defined for data that nothing writes in a kernel's lifetime, so the
serving kernels, which read one another's results, use none.  Host-side check
of the sources."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_psa_b200",
                    "csrc")


@pytest.mark.parametrize("name", ["decode.cu", "weight.cu", "evict.cu"])
def test_no_non_coherent_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    assert "grid_dep_wait()" in src
    assert "__ldg(" not in src and "ld.global.nc" not in src
    assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", src)
