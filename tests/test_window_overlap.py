"""kvq_decode_attention_window refuses outputs that share memory with one another or
with an input, on the host and before any CUDA call; out may be q itself."""
import ctypes

import pytest

import bit_mixed_precision_kvq_gb300 as kvq
from bit_mixed_precision_kvq_gb300 import build_native

B, H_q, N_Q = 2, 8, 4
FAR = 1 << 44
HEADS, ROWS = B * N_Q * H_q * 256, B * N_Q * H_q * 4  # bytes of q and out, of lse
CACHE, Q, LEN, OUT, LSE = FAR, 2 * FAR, 3 * FAR, 4 * FAR, 5 * FAR


@pytest.fixture(scope="module")
def lib():
    build_native.build()
    return kvq.load()


def layout():
    return kvq.cache_layout(B, H_q, 4, 128, 256, 10, 200, 4, 4, 32, [1])


def call(lib, L, n_q=N_Q, **kw):
    a = dict(cache=CACHE, q=Q, seq=LEN, out=OUT, lse=LSE, T=220)
    a.update(kw)
    return lib.kvq_decode_attention_window(ctypes.byref(L), a["cache"], a["q"], n_q, a["seq"], a["T"], 4, 64, 0.1, a["out"], a["lse"], None)


TOTAL = "total"
BAD = [
    dict(out=CACHE), dict(out=(CACHE, TOTAL, -256)), dict(out=CACHE - HEADS + 16), dict(out=LEN), dict(out=LEN - HEADS + 16), dict(seq=OUT + HEADS - 4),
    dict(out=Q + 16), dict(out=Q + HEADS - 16), dict(out=Q - 256), dict(out=Q - HEADS + 16),
    dict(lse=OUT), dict(lse=OUT + HEADS - 4), dict(lse=OUT - ROWS + 4), dict(lse=CACHE + 1024), dict(lse=(CACHE, TOTAL, -4)), dict(lse=CACHE - ROWS + 4),
    dict(lse=Q), dict(lse=Q + HEADS - 4), dict(lse=Q - ROWS + 4), dict(lse=LEN), dict(lse=LEN + 4), dict(lse=LEN - ROWS + 4),
    dict(out=Q, lse=Q), dict(out=Q, q=Q, seq=Q + 64),
]


@pytest.mark.parametrize("bad", BAD, ids=lambda x: str(x)[:50])
def test_overlaps_are_refused(lib, bad):
    L = layout()
    at = {k: v[0] + int(L.total_bytes) + v[2] if isinstance(v, tuple) else v for k, v in bad.items()}
    assert call(lib, L, **at) == 1


NEXT_TO = [
    dict(), dict(out=Q), dict(out=Q + HEADS), dict(out=Q - HEADS), dict(lse=OUT + HEADS), dict(lse=OUT - ROWS), dict(seq=OUT + HEADS), dict(seq=LSE - 8),
    dict(out=CACHE - HEADS), dict(out=(CACHE, TOTAL, 0)), dict(lse=0), dict(seq=0, out=Q, lse=0),
]


@pytest.mark.parametrize("good", NEXT_TO, ids=lambda x: str(x)[:50])
def test_neighbours_pass_the_checks(lib, good):
    """A length above the most is refused behind these checks, so that nothing is launched."""
    L = kvq.cache_layout(B, H_q, 4, 128, 2 ** 31 - 1, 0, 2 ** 31 - 2 ** 17, 4, 4, 32, [1])
    at = {k: v[0] + int(L.total_bytes) + v[2] if isinstance(v, tuple) else v for k, v in good.items()}
    assert int(L.total_bytes) < FAR and call(lib, L, T=2 ** 31 - 1, **at) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("B_,H_kv,n_q,T,window", [(1, 4, 1, 980, 700), (1, 4, 8, 980, 700), (40, 16, 2, 300, 120), (3, 4, 5, 400, 64)])
def test_window_in_place(cuda_dev, kvq, B_, H_kv, n_q, T, window):
    """out is q: units of one CTA and of several, one and two tiles of columns."""
    import torch
    from gpu_helpers import Case
    from serving_ref import Filled, bf16
    c = Case(B_, 28 if H_kv == 4 else 32, H_kv, T + 20, 14, T - 60, 4, 2, 64, [0])
    f = Filled(c, 90, cuda_dev)
    q = bf16((B_, n_q, c.H_q, 128), 91, cuda_dev)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=cuda_dev)
    kvq.decode_attention_window(f.L, f.cache, q, T, 20, window, out, None, lse)
    for _ in range(5):
        x, l = q.clone(), torch.empty_like(lse)
        kvq.decode_attention_window(f.L, f.cache, x, T, 20, window, x, None, l)
        assert torch.equal(x, out) and torch.equal(l, lse)
