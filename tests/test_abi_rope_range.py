"""Host-side: rotary configurations whose numbers binary32 or binary64 cannot form are refused."""
import ctypes

import pytest

from speculative_decoding_verification_91_b200 import binding as B
from speculative_decoding_verification_91_b200 import build

from .test_abi_qcache import FAKE, cache, rope


@pytest.mark.parametrize("kw", [
    dict(magnitude=1e39), dict(magnitude=1e-39), dict(magnitude=5e-324),        # cosines times it: binary32
    dict(scaling=2, theta=1e300, factor=1e10), dict(scaling=2, theta=10000.0, factor=1e305)])   # base x S^..
def test_numbers_out_of_range_are_refused(kw):
    build.build()
    lib = B.lib()
    r, out = rope(**kw), (ctypes.c_double * 128)()
    assert lib.spec_rope_frequencies(ctypes.byref(r), 128, out) == B.SPEC_EINVAL
    # (n_rows = 0 is refused too: nothing would be launched on these addresses in any case)
    assert lib.spec_rope(ctypes.byref(r), B.SPEC_BF16, FAKE, 256, 128, FAKE, 256, 128, FAKE, 0, 2, 128, 0,
                         None) == B.SPEC_EINVAL
    assert lib.spec_qcache_write(ctypes.byref(cache()), ctypes.byref(r), FAKE, 4, FAKE, 1, 0, FAKE, 256, FAKE,
                                 256, FAKE, 1 << 20, None) == B.SPEC_EINVAL


@pytest.mark.parametrize("kw", [dict(magnitude=3e38), dict(magnitude=2e-38), dict(scaling=2, theta=1e200, factor=1e100)])
def test_the_ends_of_the_ranges_are_taken(kw):
    build.build()
    out = B.spec_rope_frequencies(rope(**kw), 128)
    assert out[0] == 1.0 and all(0 <= x <= 1 for x in out)
