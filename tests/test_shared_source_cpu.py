"""What the shared-prefix kernels may not say in their source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_compression_hkv_b200", "csrc")


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "shared*.cu*"))), ids=os.path.basename)
def test_no_promise_of_unchanging_data(path):
    """These kernels are launched as programmatic dependents: they begin before
    the grids whose results they read have ended, so no load may be declared to
    be of data that stay the same while the kernel lives."""
    code = re.sub(r"//[^\n]*", "", open(path).read())
    assert not re.search(r"__ldg\s*\(|__restrict__|ld\.global\.nc", code)
