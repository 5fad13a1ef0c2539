"""Properties of the kernel sources that no run shows: what holds by luck in one
build may not hold in the next."""

import glob
import os
import re

import block_sparse_attention_sparge_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")


def test_device_arrays_state_an_alignment():
    """A device array is read in vectors of 16 bytes, so its alignment is stated:
    an element's own would put it at any multiple of four."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for line in open(path):
            if re.match(r"^(static )?__(device|constant)__ [^(]*(\([0-9]+\)[^(]*)?\[.*\];", line):
                align = re.search(r"__align__\((\d+)\)", line)
                found.append((os.path.basename(path), line.strip(),
                              int(align.group(1)) if align else 0))
    assert len(found) >= 2  # the zeros of resnorm.cu, the scratch of mask_noalloc.cu
    assert not [f for f in found if f[2] < 16]


def test_sample_offsets_into_the_grid_are_64_bits():
    """B * N goes to 2^30 - 1, so with one token a sample 3 * b passes 2^31 (where
    a 32-bit product would read in front of the grid): nothing that a run on
    tensors of ordinary size shows."""
    text = open(os.path.join(CSRC, "heads.cu")).read()
    reads = re.findall(r"p\.grid\s*[\[+][^;]*;", text)
    assert reads
    for r in reads:
        assert "int64_t" in r, r
