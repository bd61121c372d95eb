"""Host-side checks of the rotary operator and the 8-bit cache: what is refused
before any launch, and the frequencies the host forms."""
import ctypes
import math

import numpy as np
import pytest

from oracle import qcache as Q
from speculative_decoding_verification_91_b200 import binding as B
from speculative_decoding_verification_91_b200 import build

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def rope(**kw):
    a = dict(layout=B.SPEC_ROPE_HALF, span=128, n_rot=64, scaling=B.SPEC_ROPE_PLAIN, theta=10000.0, factor=1.0,
             original=0.0, turns_lo=1.0, turns_hi=32.0, magnitude=1.0)
    a.update(kw)
    return B.SpecRope(*a.values())


def cache(**kw):
    a = dict(head_dim=128, n_kv_heads=2, num_pages=10, page_size=64, block_tokens=64, split_tokens=256,
             k_pool=FAKE, v_pool=FAKE, k_scale=FAKE, v_scale=FAKE)
    a.update(kw)
    return B.SpecQCache(*a.values())


@pytest.mark.parametrize("scaling,kw", [
    ("plain", {}), ("linear", dict(factor=4.0)), ("raised", dict(factor=8.0)),
    ("parts", dict(factor=16.0, original=4096.0)),
    ("parts", dict(factor=2.5, original=8192.0, turns_lo=1.0, turns_hi=4.0))])
@pytest.mark.parametrize("span,n_rot", [(128, 64), (40, 20), (128, 16), (4, 2)])
def test_frequencies(lib, scaling, kw, span, n_rot):
    kinds = {"plain": 0, "linear": 1, "raised": 2, "parts": 3}
    got = B.spec_rope_frequencies(rope(span=span, n_rot=n_rot, scaling=kinds[scaling], theta=500000.0, **kw), 128)
    want = Q.rope_frequencies(span, n_rot, 500000.0, scaling, **kw)
    assert np.allclose(got, want, rtol=1e-14, atol=0)


@pytest.mark.parametrize("kw", [
    dict(layout=2), dict(layout=-1), dict(span=0), dict(span=127), dict(span=130), dict(n_rot=65), dict(n_rot=-1),
    dict(scaling=4), dict(scaling=-1), dict(theta=0.0), dict(theta=math.nan), dict(theta=math.inf),
    dict(magnitude=0.0), dict(magnitude=math.nan), dict(scaling=1, factor=0.5), dict(scaling=1, factor=math.inf),
    dict(scaling=2, factor=2.0, span=2, n_rot=1), dict(scaling=3, factor=2.0),
    dict(scaling=3, factor=2.0, original=100.0, turns_lo=4.0, turns_hi=4.0),
    dict(scaling=3, factor=2.0, original=100.0, turns_lo=-1.0),
    dict(scaling=3, factor=2.0, original=math.nan)])
def test_bad_rotary_configurations_are_refused(lib, kw):
    r = rope(**kw)
    out = (ctypes.c_double * 128)()
    assert lib.spec_rope_frequencies(ctypes.byref(r), 128, out) == B.SPEC_EINVAL
    assert lib.spec_rope(ctypes.byref(r), B.SPEC_BF16, FAKE, 256, 128, FAKE, 256, 128, FAKE, 4, 2, 128, 0,
                         None) == B.SPEC_EINVAL
    assert lib.spec_qcache_write(ctypes.byref(cache()), ctypes.byref(r), FAKE, 4, FAKE, 1, 4, FAKE, 256, FAKE,
                                 256, FAKE, 1 << 20, None) == B.SPEC_EINVAL


def test_rope_refusals(lib):
    def call(r=rope(), dtype=B.SPEC_BF16, x=FAKE, xr=256, xh=128, out=2 * FAKE, orow=256, oh=128, pos=FAKE, rows=4,
             heads=2, dim=128):
        return lib.spec_rope(None if r is None else ctypes.byref(r), dtype, x, xr, xh, out, orow, oh, pos, rows,
                             heads, dim, 0, None)
    for kw in (dict(r=None), dict(x=None), dict(out=None), dict(pos=None), dict(rows=0), dict(heads=0),
               dict(dtype=3), dict(dtype=-1), dict(dim=0), dict(dim=257), dict(dim=64), dict(x=FAKE + 1),
               dict(out=2 * FAKE + 1), dict(dtype=B.SPEC_FP32, x=FAKE + 2), dict(xr=-256), dict(oh=-128),
               dict(orow=0), dict(oh=64), dict(orow=255), dict(x=FAKE, out=FAKE, xr=512)):
        assert call(**kw) == B.SPEC_EINVAL, kw


def test_cache_refusals(lib):
    def write(c=cache(), table=FAKE, pages=4, lens=FAKE, B_=1, n=4, k=FAKE, kr=256, v=FAKE, vr=256, ws=FAKE,
              nbytes=1 << 20):
        return lib.spec_qcache_write(None if c is None else ctypes.byref(c), None, table, pages, lens, B_, n, k, kr,
                                     v, vr, ws, nbytes, None)

    def attn(c=cache(), q=FAKE, qr=512, heads=4, table=FAKE, pages=4, lens=FAKE, B_=1, n=4, off=0, extra=4,
             window=0, scale=0.0, out=FAKE, ws=FAKE, nbytes=1 << 30):
        return lib.spec_qcache_attn(None if c is None else ctypes.byref(c), None, q, qr, heads, table, pages, lens,
                                    B_, n, off, extra, window, scale, out, ws, nbytes, None)

    bad = [dict(c=None), dict(c=cache(k_pool=None)), dict(c=cache(v_scale=None)), dict(c=cache(n_kv_heads=0)),
           dict(c=cache(num_pages=0)), dict(c=cache(split_tokens=100)), dict(c=cache(split_tokens=64)),
           dict(c=cache(split_tokens=8192)), dict(c=cache(split_tokens=-128)), dict(c=cache(k_pool=FAKE + 8)),
           dict(c=cache(k_scale=FAKE + 4)), dict(table=None), dict(lens=None), dict(pages=0), dict(B_=0),
           dict(ws=None), dict(nbytes=100), dict(ws=FAKE + 16)]
    for kw in bad + [dict(n=-1), dict(n=65537), dict(k=None), dict(v=None), dict(kr=248), dict(vr=255), dict(kr=260),
                     dict(k=FAKE + 8)]:
        assert write(**kw) == B.SPEC_EINVAL, kw
    for kw in bad + [dict(q=None), dict(out=None), dict(n=0), dict(n=257), dict(heads=3), dict(heads=0),
                     dict(off=-1), dict(extra=-1), dict(off=65537), dict(window=-1), dict(scale=-1.0),
                     dict(scale=math.nan), dict(scale=math.inf), dict(qr=504), dict(qr=516), dict(q=FAKE + 8),
                     dict(out=FAKE + 8)]:
        assert attn(**kw) == B.SPEC_EINVAL, kw
    for c in (cache(head_dim=64), cache(page_size=32), cache(block_tokens=8), cache(num_pages=1 << 25)):
        assert write(c=c) == B.SPEC_EUNSUPPORTED and attn(c=c) == B.SPEC_EUNSUPPORTED
    assert write(n=0) == B.SPEC_OK                                     # nothing to store: nothing launched
    assert attn(c=cache(split_tokens=128), pages=1 << 20) == B.SPEC_EUNSUPPORTED     # more splits than are joined


def test_workspace_sizes(lib):
    c = cache()
    assert B.spec_qcache_write_workspace_bytes(c, 8, 5) >= 4096
    assert B.spec_qcache_write_workspace_bytes(c, 0, 5) == 0
    assert B.spec_qcache_write_workspace_bytes(None, 1, 5) == 0
    w = B.spec_qcache_attn_workspace_bytes(c, 8, 8, 5, 100)
    assert w > 4096 and B.spec_qcache_attn_workspace_bytes(c, 8, 16, 5, 100) > w
    assert B.spec_qcache_attn_workspace_bytes(c, 8, 8, 5, 100, 64) < w          # a window touches few splits
    assert B.spec_qcache_attn_workspace_bytes(c, 7, 8, 5, 100) == 0
    assert B.spec_qcache_attn_workspace_bytes(c, 8, 8, 257, 100) == 0
    assert B.spec_qcache_attn_workspace_bytes(cache(head_dim=96), 8, 8, 5, 100) == 0


def test_counts_past_32_bits_are_refused(lib):
    """Key blocks of all row blocks, and rows by query heads, are counted in 32 bits: sizes past that
    have no workspace; large ones within it do, whatever the window leaves of them."""
    c = cache()
    assert B.spec_qcache_attn_workspace_bytes(c, 8, 64, 17, 1 << 17, 64) > 4096
    assert B.spec_qcache_attn_workspace_bytes(c, 8, 65535, 17, 1 << 17, 64) == 0
    # G query heads a KV head (two of them): 17 G rows by G, below 2^32 up to G = 15894
    assert B.spec_qcache_attn_workspace_bytes(c, 2 * 15894, 1, 17, 100) > 4096
    assert B.spec_qcache_attn_workspace_bytes(c, 2 * 15895, 1, 17, 100) == 0


@pytest.mark.parametrize("n", [17, 100, 256])
def test_a_workspace_serves_smaller_calls(lib, n):
    """The size for the largest call covers smaller ones, which take the cache's own, shorter splits."""
    for c in (cache(), cache(split_tokens=128), cache(block_tokens=16)):
        for heads in (8, 64):
            most = B.spec_qcache_attn_workspace_bytes(c, heads, 8, n, 400)
            for batch, rows, pages in ((8, 17, 400), (8, 1, 400), (1, 17, 400), (3, 5, 37), (1, 1, 1)):
                assert B.spec_qcache_attn_workspace_bytes(c, heads, batch, rows, pages) <= most
