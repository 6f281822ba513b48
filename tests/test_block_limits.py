"""Limits of prompt attention over caches with block scales, told before any device call (CPU)."""
import pytest
import torch

import fp8_paged_kv_gb300 as fpk

A = 1 << 20  # a 256-byte aligned address that is never followed

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="run where no device is visible")


@host_only
@pytest.mark.parametrize("page_size", [16, 48, 256])
def test_tables_of_2_31_tokens(page_size):
    """A context that could be longer than 2^31 - 128 tokens does not round up to blocks in 31 bits."""
    from fp8_paged_kv_gb300 import build
    build.build()
    lib = fpk.load_library()

    def call(max_pages, cu=A):
        return lib.fpk_paged_prefill_attn_fp8_block(A, cu, 4, A, A, A, max_pages, A, None, 0, A, None, A, 1 << 40, 0.1, 1, 1, 1, 128,
                                                    page_size, 8, None)

    most = ((1 << 31) - 128) // page_size
    for pages in (most + 1, (1 << 31) // page_size, (1 << 31) - 1):
        assert call(pages) == fpk.FPK_EUNSUPPORTED, pages
    # (a missing pointer is told behind the limits: this many pages are within them)
    assert call(most, cu=None) == fpk.FPK_EINVAL
