"""Sizes of the block-cache operators whose products do not fit 64 bits: refused before any CUDA call (fake addresses)."""

import pytest

from test_block_cache_host import UNSUPPORTED, Call, built_library, refused  # noqa: F401


@pytest.mark.parametrize("B,Nkv", [(1 << 62, 4), (1 << 61, 8), (1 << 32, 1 << 16), (65536, 1)])
def test_batches_beyond_any_memory(B, Nkv):
    """B Nkv, and with it every size, may be 0 in 64 bits."""
    c = Call(B=B, N=Nkv, Nkv=Nkv, S=1, H=16, C=32)
    refused(c.size, UNSUPPORTED)
    refused(lambda: c.forward(1 << 20, 1 << 40), UNSUPPORTED)
    refused(c.evict, UNSUPPORTED)
