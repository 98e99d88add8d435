"""What the paged cache's kernels may not contain, looked up in their sources."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "flashattention_backward_gb300", "csrc")


@pytest.mark.parametrize("name", ["fa_paged.cuh", "fa_decode.cuh", "fa_decode.cu", "fa_decode_fp32.cu", "fa_cache.cu",
                                  "fa_pages.cu"])
def test_early_kernels_read_coherently(name):
    """These kernels are on the GPU before the work in front of them has ended.  A non-coherent load promises data that
    does not change while the kernel runs, and may be moved in front of the wait for that work."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg\s*\(|ld\.global[.\w]*\.nc|__restrict__", code)
