"""How the attention over the paged cache divides its keys, on the host: every
row tile, of whatever length, gets splits that hold its keys and that the grid,
the cluster and the workspace have room for."""
import itertools

import pytest

import clustered_multipole_approximation_b200 as muse
from clustered_multipole_approximation_b200 import build
from clustered_multipole_approximation_b200.kv_cache import muse_cache, muse_cache_division, muse_cache_index, muse_strides

FAKE = 0x1000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return muse.load_library()


def lengths(cap):
    some = {0, 1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, cap // 3, cap // 2, cap - 1, cap}
    return sorted(x for x in some if 0 <= x <= cap)


@pytest.mark.parametrize("dtype,cache", [(0, 0), (0, 2), (0, 3), (0, 1), (1, 1), (1, 0), (1, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_every_length_has_its_splits(lib, dtype, cache, D):
    scale = FAKE if cache >= 2 else None
    for (B, Hkv), G, n, (page, wide), window in itertools.product(
            [(1, 1), (1, 2), (2, 1), (1, 8), (3, 5), (64, 8), (40, 16)], [1, 3, 8], [1, 5, 40, 300, 2048],
            [(1, 1), (16, 2), (16, 64), (24, 100), (16, 1024), (256, 256), (64, 1 << 14), (1024, 1 << 20)],
            [0, 1, 300, 5000, 1 << 30]):
        sh = muse.muse_shape(B, Hkv * G, Hkv, n, D, dtype, 0)
        ca = muse_cache(FAKE, FAKE, scale, scale, 64, page, cache)
        ix = muse_cache_index(FAKE, FAKE, None, wide)
        size = lib.muse_attn_cache_workspace_size(sh, ca, ix)
        assert size > 0
        what = (B, Hkv, G, n, page, wide, window)
        for length in lengths(page * wide):
            d = muse_cache_division()
            assert lib.muse_debug_cache_division(sh, ca, ix, window, length, d) == 0
            assert d.keys > 0 and d.keys % d.quantum == 0, what
            assert 1 <= d.parts <= d.splits and d.tiles * d.splits < 1 << 31, what
            assert d.parts * d.keys >= length and (d.parts == 1 or (d.parts - 1) * d.keys < length), what
            if d.splits > 1 and not d.cluster:  # partial rows, maxima and sums
                assert size >= d.tiles * d.splits * d.rows * (D * 4 + 8), what
            assert not d.cluster or d.splits <= 8, what


def test_writes_and_reads_need_no_query_heads(lib):
    """Hq = 0, and a number of q-heads whose rows alone would be too many, pass the
    shape's checks (an unknown cache dtype, checked later, is what is refused)."""
    ca, ix = muse_cache(FAKE, FAKE, None, None, 4, 16, 9), muse_cache_index(FAKE, FAKE, None, 2)
    st = muse_strides(384, 192, 64)
    for Hq in (0, 2, 1 << 30):
        sh = muse.muse_shape(2, Hq, 2, 3, 64, 0, 0)
        assert lib.muse_cache_write(FAKE, st, FAKE, st, sh, ca, ix, None, None) == 1
        assert b"cache dtype" in lib.muse_last_error()
        assert lib.muse_cache_read(FAKE, FAKE, sh, ca, ix, None, None, None) == 1
        assert b"cache dtype" in lib.muse_last_error()
    sh = muse.muse_shape(2, 0, 2, 3, 64, 0, 0)
    assert lib.muse_attn_cache(FAKE, st, FAKE, st, None, sh, ca, ix, 1.0, 1, 0, None, FAKE, 1 << 40, None) == 1
    assert b"Hq" in lib.muse_last_error()


def test_buffers_that_share_memory_are_refused(lib):
    """K and V of a read, and the caches and scales of a write, over the same memory
    or a part of it."""
    far = 1 << 40
    sh, ix, st = muse.muse_shape(2, 2, 2, 3, 64, 0, 0), muse_cache_index(FAKE, FAKE, None, 2), muse_strides(384, 192, 64)
    ca = muse_cache(FAKE, far, None, None, 4, 16, 0)
    size = 2 * 2 * 3 * 64 * 2
    for v in (FAKE, FAKE + size - 16, FAKE - size + 16):
        assert lib.muse_cache_read(FAKE, v, sh, ca, ix, None, None, None) == 1
        assert b"share" in lib.muse_last_error(), v
    cells = 4 * 2 * 16
    other = muse_strides(384, 64, 128)
    for dt, bytes_ in ((0, 2), (1, 4)):
        for v in (FAKE, FAKE + cells * 64 * bytes_ - 16):
            for V, vs in ((far, st), (FAKE, other)) if v == FAKE else ((FAKE, st),):
                ca = muse_cache(FAKE, v, None, None, 4, 16, dt)
                assert lib.muse_cache_write(FAKE, st, V, vs, sh, ca, ix, None, None) == 1
                assert b"share" in lib.muse_last_error()
    for v, vs_ in ((FAKE + cells * 64 - 16, far), (far, FAKE), (far, FAKE + 4 * cells - 4)):
        ca = muse_cache(FAKE, v, FAKE, vs_, 4, 16, 3)
        assert lib.muse_cache_write(FAKE, st, far, st, sh, ca, ix, None, None) == 1
        assert b"share" in lib.muse_last_error()


def test_refusals(lib):
    sh, ca, ix = muse.muse_shape(1, 1, 1, 1, 64, 0, 0), muse_cache(FAKE, FAKE, None, None, 4, 16, 0), \
        muse_cache_index(FAKE, FAKE, None, 2)
    d = muse_cache_division()
    f = lib.muse_debug_cache_division
    assert f(sh, ca, ix, 0, 32, d) == 0
    assert f(sh, ca, ix, 0, 33, d) == 1 and f(sh, ca, ix, 0, -1, d) == 1 and f(sh, ca, ix, -1, 1, d) == 1
    assert f(sh, ca, ix, 0, 1, None) == 1 and f(None, ca, ix, 0, 1, d) == 1
