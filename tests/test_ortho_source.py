"""A property of the chained kernels that no run shows: each is on the machine before the one
before it has ended, so what that one (or the kernel itself) writes is not read through the
read-only path, which holds for memory that nobody writes while the kernel is there."""

import os
import re

import block_sparse_attention_sparge_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")


def test_no_read_only_loads_of_what_the_chain_writes():
    text = open(os.path.join(CSRC, "ortho.cu")).read()
    assert "grid_wait();" in text
    assert not re.findall(r"__ldg\(|ldg_no_l1\(|[^_]load8\(|ld\.global\.nc", text)
