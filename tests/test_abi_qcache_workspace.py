"""Host-side: workspace sizes of the 8-bit attention at the ends of their ranges."""
import ctypes

import pytest

from speculative_decoding_verification_91_b200 import binding as B
from speculative_decoding_verification_91_b200 import build

from .test_abi_qcache import FAKE, cache


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return B.lib()


def refused_for_size(lib, c, heads, n, pages, window, nbytes):
    """Whether a call of one sequence is refused because its workspace is too small (nothing is launched:
    the sizes given are too small for every call)."""
    return lib.spec_qcache_attn(ctypes.byref(c), None, FAKE, heads * 128, heads, FAKE, pages, FAKE, 1, n, 0, n, window,
                                0.0, FAKE, FAKE, nbytes, None) == B.SPEC_EINVAL


@pytest.mark.parametrize("split", [128, 256, 1024])
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("window", [0, 1 << 24])
def test_prompt_chunks_over_tables_too_wide_for_single_rows(lib, split, block, window):
    """A prompt chunk takes longer splits than a verify step, and so wider tables: what the call accepts has a
    size, and that size still covers the verify steps that fit."""
    c = cache(split_tokens=split, block_tokens=block)
    most = 8192 * split // 64                            # pages of 8192 splits
    for pages in (most, most + 1, 3 * most):
        for n in (18, 256):
            assert refused_for_size(lib, c, 8, n, pages, window, 5000)
            size = B.spec_qcache_attn_workspace_bytes(c, 8, 1, n, pages, window)
            assert size > 4096
            for rows in (1, 17):
                assert size >= B.spec_qcache_attn_workspace_bytes(c, 8, 1, rows, most, window) > 4096
        assert (B.spec_qcache_attn_workspace_bytes(c, 8, 1, 17, pages, window) > 0) == (pages == most)
