"""The eviction writes the new lengths while it still reads the old ones, so the two must not share memory: the call
refuses that before anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    import paged_kv_cache_kvh_gb300 as pkv
    return pkv._lib


def _call(lib, lens, new_lens, n=4):
    at = ctypes.c_void_p
    return lib.pkv_evict_kvcache(at(4096), at(4096), at(4096), 16, at(4096), 16, at(lens), n, 8, 128, 256, 4096, 300, 4, 32,
                                 at(8192), 2, at(4096), at(new_lens), None)


@pytest.mark.parametrize("apart", [0, 4, 8, 12, -4, -12])
def test_lengths_that_overlap_are_refused(lib, apart):
    assert _call(lib, 1 << 20, (1 << 20) + apart) == -6


def test_longer_calls_overlap_farther_apart(lib):
    assert _call(lib, 1 << 20, (1 << 20) + 16, n=5) == _call(lib, 1 << 20, (1 << 20) - 16, n=5) == -6
    assert _call(lib, 1 << 20, (1 << 20) + 4, n=0) == 0
