"""What the kernels of the paged cache in 8 bits may not contain, looked up in their sources."""

import pytest

from test_paged_sources import test_early_kernels_read_coherently as reads_coherently


@pytest.mark.parametrize("name", ["fa_e4m3.cuh", "fa_cache_e4m3.cu", "fa_decode_e4m3.cu", "fa_decode_e4m3_sm103.cu"])
def test_kernels_in_8_bits_read_coherently(name):
    reads_coherently(name)
