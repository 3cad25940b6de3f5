"""What the Python binding of the serving calls checks of a workspace and of
its integers, before the C call sees them (no GPU: the current device and the
library are stood in for)."""
import types

import pytest

import bit_mixed_precision_kvq_gb300 as kvq
from bit_mixed_precision_kvq_gb300 import build_native

FAKE, FAR = 1 << 40, 1 << 44


class Elsewhere:
    """A tensor as the binding looks at it, on a device of choice."""

    def __init__(self, dev=0, numel=1 << 24, contiguous=True):
        self._dev, self._numel, self._contiguous = dev, numel, contiguous

    def get_device(self):
        return self._dev

    def is_contiguous(self):
        return self._contiguous

    def numel(self):
        return self._numel

    def element_size(self):
        return 1

    def data_ptr(self):
        return FAR


@pytest.fixture
def L(monkeypatch):
    """CPU tensors count as on the current device (get_device() == -1), and
    calls are recorded."""
    import torch
    build_native.build()
    lay = kvq.cache_layout(2, 8, 4, 128, 256, 10, 200, 4, 4, 32, [1])
    smaller = kvq.cache_layout(2, 8, 4, 128, 150, 10, 110, 4, 4, 32, [1])
    calls = []

    def record(*a):
        calls.append(a)
        return 0

    names = ("kvq_decode_attention_tree", "kvq_tree_commit", "kvq_attention_mass", "kvq_cache_evict")
    monkeypatch.setattr(kvq, "load", lambda: types.SimpleNamespace(**{n: record for n in names}))
    monkeypatch.setattr(kvq, "_current", lambda stream: (torch, -1, 0))
    lay.calls, lay.smaller = calls, smaller
    return lay


def _tree(L, ws, T=220, **kw):
    import torch
    q = torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16)
    kd = torch.zeros(2, 4, 3, 128, dtype=torch.bfloat16)
    kvq.decode_attention_tree(L, FAKE, q, kd, kd, torch.zeros(2, 3, dtype=torch.int64), T, q, workspace=ws, **kw)


def test_tree_workspace_is_checked(L):
    for dev in (0, 1, 3):   # another device than the current one
        with pytest.raises(ValueError, match="device"):
            _tree(L, Elsewhere(dev))
    with pytest.raises(ValueError, match="contiguous"):
        _tree(L, Elsewhere(-1, contiguous=False))
    for n in (101, -1):     # more bytes than there are
        with pytest.raises(ValueError, match="bytes"):
            _tree(L, Elsewhere(-1, 100), ws_bytes=n)
    assert not L.calls
    _tree(L, Elsewhere(-1, 100))
    _tree(L, Elsewhere(-1, 100), ws_bytes=64)
    _tree(L, FAR, ws_bytes=77)
    _tree(L, None)
    assert [c[-3:-1] for c in L.calls] == [(FAR, 100), (FAR, 64), (FAR, 77), (0, 0)]


def test_integers_are_converted_or_refused(L):
    """Whole numbers of other types are taken, and what an int32 does not
    hold is refused and not cut to 32 bits."""
    import numpy as np
    import torch
    mass = torch.zeros(2, 4, 256)
    i32 = dict(dtype=torch.int32)
    kd = torch.zeros(2, 4, 3, 128, dtype=torch.bfloat16)
    lse, q = torch.zeros(2, 3, 8), torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16)

    def calls(T, T_dst=120, recent=4):
        yield lambda: _tree(L, Elsewhere(-1), T)
        yield lambda: kvq.tree_commit(L, FAKE, kd, kd, torch.zeros(2, 2, **i32), torch.zeros(2, **i32), T)
        yield lambda: kvq.attention_mass(L, FAKE, q, lse, T, mass)
        yield lambda: kvq.cache_evict(L, FAKE, mass, T, L.smaller, FAR, T_dst, torch.zeros(2, 4, int(T_dst), **i32), recent)

    for T in (2 ** 32 + 220, -2 ** 31 - 1):
        for f in calls(T):
            with pytest.raises(ValueError, match="int32"):
                f()
    for kw in (dict(recent=2 ** 32 + 4),):
        with pytest.raises(ValueError, match="int32"):
            list(calls(220, **kw))[-1]()
    assert not L.calls
    for T in (220, np.int64(220), torch.tensor(220)):
        for f in calls(T, np.int32(120), np.int64(4)):
            f()
    assert len(L.calls) == 12
    for c in L.calls:
        assert all(type(x) in (int, float) or "Layout" in str(type(x)) or "byref" in str(type(x)) or "CArg" in str(type(x))
                   for x in c), [type(x) for x in c]
