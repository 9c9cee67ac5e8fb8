"""CPU: dynamic LDS arrays state an alignment.  They follow a kernel's other LDS
variables; without one an array starts where its element type may, and reads of
four words at a time, or of words in a char array, are undefined there."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_gradient_backward_amd", "csrc")


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "lm_*.hip"))), ids=os.path.basename)
def test_dynamic_lds_is_aligned(path):
    text = open(path).read()
    arrays = re.findall(r"extern __shared__([^;]*);", text)
    wide = [a for a in arrays if "aligned(16)" not in a]
    # the sums' bits are words and read as words or bytes
    assert [a.strip() for a in wide] in ([], ["uint32_t bits[]"])
