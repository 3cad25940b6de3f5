"""Lengths whose tiles would pass 32 bits are refused on the host, before any
CUDA call (the addresses are never dereferenced)."""
import ctypes

import pytest

import bit_mixed_precision_kvq_gb300 as kvq
from bit_mixed_precision_kvq_gb300 import build_native

FAKE, FAR = 1 << 44, 1 << 50   # farther apart than a cache of 2^31 positions is long
MOST = 2 ** 31 - 2 ** 16


@pytest.fixture(scope="module")
def lib():
    build_native.build()
    return kvq.load()


def _layout(T_cap, vis_end):
    return kvq.cache_layout(1, 1, 1, 128, T_cap, 0, vis_end, 2, 2, 128)


@pytest.mark.parametrize("T", [MOST + 1, 2 ** 31 - 200, 2 ** 31 - 1])
def test_lengths_past_the_last_tile(lib, T):
    L, S = _layout(2 ** 31 - 1, 2 ** 31 - 2 ** 17), _layout(4096, 1024)
    ref = ctypes.byref
    assert lib.kvq_decode_attention_tree(ref(L), FAKE, FAR, 2 * FAR, 3 * FAR, 256, 256, 128, 2, 4 * FAR, 0, None, T, 0.1,
                                         5 * FAR, None, 6 * FAR, 1 << 40, None) == 2
    assert lib.kvq_attention_mass(ref(L), FAKE, FAR, 2 * FAR, 1, None, T, None, 0, None, 0.1, None, 1.0, 5 * FAR, None) == 2
    assert lib.kvq_cache_evict(ref(L), FAKE, FAR, None, T, ref(S), 2 * FAR, 2048, 1, 3 * FAR, None, None, None) == 2


def test_capacity_past_the_last_stride(lib):
    """The zeros behind the kept masses go to the new cache's capacity."""
    L, S = _layout(2 ** 31 - 1, 4096), _layout(2 ** 31 - 1, 1024)
    assert lib.kvq_cache_evict(ctypes.byref(L), FAKE, FAR, None, 5000, ctypes.byref(S), 2 * FAR, 2048, 1, 3 * FAR, 4 * FAR,
                               None, None) == 2
