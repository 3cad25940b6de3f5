"""Eviction refuses outputs that share memory with one another or with what it
reads (on the host, before any CUDA call: the addresses are never
dereferenced)."""
import ctypes

import pytest

import bit_mixed_precision_kvq_gb300 as kvq
from bit_mixed_precision_kvq_gb300 import build_native

FAR = 1 << 44
B, H, T_CAP, T_CAP_DST, T_DST = 2, 4, 256, 150, 120


@pytest.fixture(scope="module")
def lib():
    build_native.build()
    return kvq.load()


def _call(lib, **at):
    L = kvq.cache_layout(B, 8, H, 128, T_CAP, 10, 200, 4, 4, 32, [1])
    D = kvq.cache_layout(B, 8, H, 128, T_CAP_DST, 10, 110, 4, 4, 32, [1])
    a = dict(cache=FAR, mass=2 * FAR, seq_len=3 * FAR, cache_dst=4 * FAR, keep=5 * FAR, mass_dst=6 * FAR, new_len=7 * FAR)
    size = dict(cache=int(L.total_bytes), mass=4 * B * H * T_CAP, seq_len=4 * B, cache_dst=int(D.total_bytes),
                keep=4 * B * H * T_DST, mass_dst=4 * B * H * T_CAP_DST, new_len=4 * B)
    a.update({k: f(a, size) for k, f in at.items()})
    return lib.kvq_cache_evict(ctypes.byref(L), a["cache"], a["mass"], a["seq_len"], 220, ctypes.byref(D), a["cache_dst"],
                               T_DST, 4, a["keep"], a["mass_dst"], a["new_len"], None)


PAIRS = [(w, o) for w in ("keep", "mass_dst", "new_len") for o in ("cache", "mass", "seq_len", "cache_dst", "keep", "mass_dst")
         if w != o]


@pytest.mark.parametrize("out,other", PAIRS)
def test_outputs_share_no_memory(lib, out, other):
    assert _call(lib, **{out: lambda a, n: a[other]}) == 1                              # the same start
    assert _call(lib, **{out: lambda a, n: a[other] + n[other] - 4}) == 1               # over its last entry
    assert _call(lib, **{out: lambda a, n: a[other] - n[out] + 4}) == 1                 # reaching into its first
