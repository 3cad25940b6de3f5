"""Refusals of the norm-and-rotation, tree-verification and windowed decode
calls: rejected on the host before any CUDA call (the addresses are never
dereferenced), and the Python binding's own checks."""
import ctypes
import types

import pytest

import bit_mixed_precision_kvq_gb300 as kvq
from bit_mixed_precision_kvq_gb300 import build_native

FAKE = 1 << 40   # far apart, so that no two buffers meet
FAR = 1 << 44


@pytest.fixture(scope="module")
def lib():
    build_native.build()
    return kvq.load()


def _layout(**kw):
    a = dict(B=2, H_q=8, H_kv=4, D=128, T_cap=256, vis_start=10, vis_end=200, k_bits=4, v_bits=4, group_size=32,
             protected=[1])
    a.update(kw)
    return kvq.cache_layout(**a)


def _rows(data, sb, sh, st):
    return kvq._ROWS(data, sb, sh, st)


def _desc(**kw):
    R = kvq.rope_desc(128, [0] * 16 + [1] * 24 + [2] * 24)
    for k, v in kw.items():
        if k == "axis0":
            R.axis[0] = v
        else:
            setattr(R, k, v)
    return R


# rows of a fused projection [B = 2][n = 6][8 + 2 * 4 heads]
FQ, FK = (FAR, 6 * 2048, 128, 2048), (FAR + 2 * 8 * 128, 6 * 2048, 128, 2048)
OQ, OK = (2 * FAR, 6 * 1024, 128, 1024), (3 * FAR, 4 * 6 * 128, 6 * 128, 128)


def _rope(lib, L=None, R=None, q=FQ, k=FK, n=6, pos=4 * FAR, pa=12, pb=6, freq=5 * FAR, wq=0, wk=0, eps=1e-6, qo=OQ, ko=OK):
    L, R = L or _layout(), R or _desc()
    rows = [None if x is None else _rows(*x) for x in (q, k, qo, ko)]
    return lib.kvq_norm_rope(ctypes.byref(L), ctypes.byref(R), rows[0], rows[1], n, pos, pa, pb, freq, wq, wk, eps, rows[2], rows[3],
                             None)


ROPE_BAD = [
    dict(q=None), dict(ko=None), dict(q=None, k=None, qo=None, ko=None), dict(q=(0,) + FQ[1:]), dict(q=(FAR + 8,) + FQ[1:]),
    dict(k=(FAR, -8, 128, 2048)), dict(k=(3 * FAR + 2 ** 30, 12288, 4, 2048)), dict(q=(FAR, 12288, 128, 2044)),
    dict(q=(FAR, 1 << 60, 128, 2048)), dict(pos=0), dict(pos=4 * FAR + 2), dict(pa=-1), dict(pb=-1), dict(pa=1 << 60), dict(freq=0),
    dict(freq=5 * FAR + 2), dict(wq=6 * FAR + 8), dict(wk=6 * FAR + 2), dict(eps=-1.0), dict(eps=float("nan")), dict(n=-1),
    # output rows that share memory: a stride of 0, rows inside one another
    dict(qo=(2 * FAR, 0, 128, 1024)), dict(qo=(2 * FAR, 6 * 1024, 128, 1016)), dict(ko=(3 * FAR, 4 * 6 * 128, 128, 128)),
    # outputs over inputs, in place apart
    dict(qo=(FAR + 256, 12288, 128, 2048)), dict(qo=(FAR, 12288, 128, 4096)), dict(ko=FQ), dict(qo=FK), dict(ko=OQ),
    dict(qo=(FAR + 4 * 256, 12288, 128, 2048), q=OQ),
    dict(pos=2 * FAR + 1024), dict(freq=3 * FAR + 512), dict(wq=2 * FAR), dict(wk=3 * FAR + 16), dict(pos=2 * FAR - 4 * 20),
    dict(R=dict(rot_dim=0)), dict(R=dict(rot_dim=136)), dict(R=dict(rot_dim=12)), dict(R=dict(interleaved=2)), dict(R=dict(n_axes=0)),
    dict(R=dict(n_axes=5)), dict(R=dict(n_axes=2)), dict(R=dict(axis0=3)),
]


@pytest.mark.parametrize("bad", ROPE_BAD, ids=lambda x: str(x)[:50])
def test_rope_argument_checks(lib, bad):
    bad = dict(bad)
    if "R" in bad:
        bad["R"] = _desc(**bad["R"])
    assert _rope(lib, **bad) == 1


def test_rope_null_arguments_and_no_tokens(lib):
    L, R, x = _layout(), _desc(), _rows(*FQ)
    assert lib.kvq_norm_rope(None, ctypes.byref(R), x, None, 1, FAR, 0, 0, FAR, 0, 0, 0.0, x, None, None) == 1
    assert lib.kvq_norm_rope(ctypes.byref(L), None, x, None, 1, FAR, 0, 0, FAR, 0, 0, 0.0, x, None, None) == 1
    assert _rope(lib, n=0) == 0
    # in place, as parts of one buffer, and one side alone pass the checks (and stop at the missing device, or run nothing)
    assert _rope(lib, n=0, qo=FQ, ko=FK) == 0


def test_rope_too_many_tokens(lib):
    L = _layout(B=64, H_q=1, H_kv=1, protected=[])
    big = 2 ** 31 // 64
    x = (FAR, big * 128, 128, 128)
    assert _rope(lib, L=L, q=x, k=None, qo=(FAR << 2, big * 128, 128, 128), ko=None, n=big, pa=0, pb=0, pos=6 * FAR) == 2


def _verify(lib, **bad):
    a = dict(B=3, n_q=5, vocab=1000, logits=FAKE, fp32=0, lsb=5000, lst=1000, tokens=FAR, mask=2 * FAR, msb=5, draft=0, dsb=0, dst=0,
             accept=3 * FAR, race=4 * FAR, temp=0, size=0, path=5 * FAR, plen=6 * FAR, next=7 * FAR, logp=0)
    a.update(bad)
    return lib.kvq_tree_verify(a["B"], a["n_q"], a["vocab"], a["logits"], a["fp32"], a["lsb"], a["lst"], a["tokens"], a["mask"], a["msb"],
                               a["draft"], a["dsb"], a["dst"], a["accept"], a["race"], a["temp"], a["size"], a["path"], a["plen"],
                               a["next"], a["logp"], None)


VERIFY_BAD = [
    (dict(B=0), 1), (dict(n_q=0), 1), (dict(n_q=65), 1), (dict(vocab=0), 1), (dict(vocab=(1 << 30) + 1), 1), (dict(fp32=2), 1),
    (dict(logits=0), 1), (dict(logits=FAKE + 1), 1), (dict(logits=FAKE + 2, fp32=1), 1), (dict(tokens=0), 1), (dict(tokens=FAR + 2), 1),
    (dict(mask=0), 1), (dict(mask=2 * FAR + 4), 1), (dict(msb=4), 1), (dict(msb=-5), 1), (dict(accept=0), 1), (dict(race=0), 1),
    (dict(race=4 * FAR + 1), 1), (dict(temp=8 * FAR + 2), 1), (dict(size=8 * FAR + 1), 1), (dict(path=0), 1), (dict(plen=0), 1),
    (dict(next=0), 1), (dict(logp=9 * FAR + 2), 1), (dict(lsb=-1), 1), (dict(lst=-1), 1), (dict(lsb=1 << 62), 1),
    (dict(draft=9 * FAR, dsb=-1), 1), (dict(draft=9 * FAR + 2), 1), (dict(draft=9 * FAR, dst=1 << 61), 1), (dict(B=65536), 2),
    # outputs over one another and over inputs
    (dict(path=6 * FAR), 1), (dict(next=6 * FAR + 8), 1), (dict(logp=5 * FAR + 56), 1), (dict(path=FAR + 56), 1), (dict(plen=2 * FAR + 8), 1),
    (dict(logp=3 * FAR), 1), (dict(next=4 * FAR + 11996), 1), (dict(plen=8 * FAR, size=8 * FAR), 1), (dict(next=8 * FAR, temp=8 * FAR + 8), 1),
    (dict(logp=FAKE + 2 * 14999), 1), (dict(logp=9 * FAR + 4 * 100, draft=9 * FAR, dsb=5000, dst=1000), 1),
]


@pytest.mark.parametrize("bad,code", VERIFY_BAD, ids=lambda x: str(x)[:50])
def test_verify_argument_checks(lib, bad, code):
    assert _verify(lib, **bad) == code


def _window(lib, L=None, **bad):
    a = dict(cache=FAKE, q=FAR, n_q=4, seq=0, T=220, sink=4, window=64, scale=0.1, out=2 * FAR, lse=0)
    a.update(bad)
    return lib.kvq_decode_attention_window(ctypes.byref(L or _layout()), a["cache"], a["q"], a["n_q"], a["seq"], a["T"], a["sink"],
                                           a["window"], a["scale"], a["out"], a["lse"], None)


WINDOW_BAD = [
    dict(cache=0), dict(cache=FAKE + 128), dict(q=0), dict(q=FAR + 8), dict(n_q=0), dict(n_q=65), dict(seq=FAR + 2), dict(T=0), dict(T=257),
    dict(T=-1), dict(sink=-1), dict(window=0), dict(window=-5), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=0),
    dict(out=2 * FAR + 2), dict(lse=3 * FAR + 1),
]


@pytest.mark.parametrize("bad", WINDOW_BAD, ids=lambda x: str(x)[:50])
def test_window_argument_checks(lib, bad):
    assert _window(lib, **bad) == 1


def test_window_lengths_past_32_bits(lib):
    L = _layout(B=1, H_q=1, H_kv=1, T_cap=2 ** 31 - 1, vis_start=0, vis_end=2 ** 31 - 2 ** 17, protected=[])
    for T in (2 ** 31 - 2 ** 16 + 1, 2 ** 31 - 1):
        assert _window(lib, L, cache=1 << 44, q=1 << 50, out=1 << 51, T=T) == 2


def test_corrupted_layouts_are_refused(lib):
    bad = kvq.Layout.from_buffer_copy(_layout())
    bad.off[2] += 256
    assert _window(lib, bad) == 1 and _rope(lib, L=bad) == 1


def test_rope_desc_checks():
    for kw in (dict(rot_dim=64, axes=[0] * 31), dict(rot_dim=4, axes=[0, 0]), dict(rot_dim=12, axes=[0] * 6), dict(rot_dim=136, axes=[0] * 68),
               dict(rot_dim=16, axes=[0] * 7 + [4]), dict(rot_dim=16, axes=[0] * 7 + [-1])):
        with pytest.raises(ValueError):
            kvq.rope_desc(**kw)
    R = kvq.rope_desc(16, [0, 2, 1, 0, 0, 0, 0, 1], True)
    assert (R.rot_dim, R.interleaved, R.n_axes, list(R.axis)[:9]) == (16, 1, 3, [0, 2, 1, 0, 0, 0, 0, 1, 0])


@pytest.fixture
def recorded(monkeypatch):
    """CPU tensors count as on the current device (get_device() == -1), and
    calls are recorded."""
    import torch
    build_native.build()
    L, calls = _layout(), []

    def record(*a):
        calls.append(a)
        return 0

    names = ("kvq_norm_rope", "kvq_tree_verify", "kvq_decode_attention_window")
    monkeypatch.setattr(kvq, "load", lambda: types.SimpleNamespace(**{n: record for n in names}))
    monkeypatch.setattr(kvq, "_current", lambda stream: (torch, -1, 0))
    return L, calls


def test_binding_of_rope(recorded):
    import torch
    L, calls = recorded
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    qkv = torch.zeros(2, 6, 16, 128, **bf)
    good = dict(L=L, R=_desc(), q=qkv[:, :, :8], k=qkv[:, :, 8:12], pos=torch.zeros(3, 2, 6, **i32), inv_freq=torch.zeros(64),
                q_out=torch.zeros(2, 6, 8, 128, **bf), k_out=torch.zeros(2, 4, 6, 128, **bf).transpose(1, 2))
    for bad in (dict(q=None), dict(k=None, q=None, k_out=None, q_out=None), dict(q=qkv[:, :, :7]), dict(q=qkv[0]), dict(k=qkv.float()[:, :, :4]),
                dict(q_out=torch.zeros(2, 5, 8, 128, **bf)), dict(k_out=torch.zeros(2, 6, 4, 256, **bf)[..., ::2]), dict(pos=torch.zeros(2, 2, 6, **i32)),
                dict(pos=torch.zeros(3, 2, 6)), dict(pos=torch.zeros(3, 6, 2, **i32)), dict(pos=torch.zeros(3, 2, 12, **i32)[..., ::2]), dict(pos=torch.zeros(6, **i32)),
                dict(inv_freq=torch.zeros(63)), dict(inv_freq=torch.zeros(64).double()), dict(q_weight=torch.zeros(128)), dict(k_weight=torch.zeros(64, **bf))):
        with pytest.raises(ValueError):
            kvq.norm_rope(**{**good, **bad})
    assert not calls
    kvq.norm_rope(**good)
    kvq.norm_rope(**{**good, "pos": torch.zeros(4, 6, **i32)})       # one row of positions for the batch; an axis more
    kvq.norm_rope(**{**good, "q": None, "q_out": None})
    unpack = __import__("struct").Struct("=Qqqq").unpack
    assert unpack(calls[0][2])[1:] == (6 * 16 * 128, 128, 16 * 128) and unpack(calls[0][-2])[1:] == (4 * 6 * 128, 6 * 128, 128)
    assert calls[0][4] == 6 and calls[0][6:8] == (12, 6) and calls[1][6:8] == (6, 0) and calls[2][2] is None
    kvq.norm_rope(**{**good, "q": qkv[:, :0, :8], "q_out": torch.zeros(2, 0, 8, 128, **bf), "k": None, "k_out": None, "pos": torch.zeros(3, 2, 0, **i32)})
    assert len(calls) == 3


def test_binding_of_verify(recorded):
    import torch
    _, calls = recorded
    i32 = dict(dtype=torch.int32)
    good = dict(logits=torch.zeros(3, 5, 100), tokens=torch.zeros(3, 5, **i32), tree_mask=torch.zeros(3, 5, dtype=torch.int64), accept=torch.zeros(3, 5),
                race=torch.zeros(3, 100), path=torch.zeros(3, 5, **i32), path_len=torch.zeros(3, **i32), next_token=torch.zeros(3, **i32))
    for bad in (dict(logits=torch.zeros(3, 5, 100).half()), dict(logits=torch.zeros(5, 100)), dict(logits=torch.zeros(3, 5, 200)[..., ::2]),
                dict(tokens=torch.zeros(3, 5, dtype=torch.int64)), dict(tokens=torch.zeros(3, 6, **i32)), dict(tree_mask=torch.zeros(2, 5, dtype=torch.int64)),
                dict(tree_mask=torch.zeros(3, 5, **i32)), dict(accept=torch.zeros(3, 4)), dict(accept=torch.zeros(3, 10)[:, ::2]), dict(race=torch.zeros(3, 99)),
                dict(race=torch.zeros(3, 100).double()), dict(path=torch.zeros(3, 4, **i32)), dict(path_len=torch.zeros(3)), dict(next_token=torch.zeros(4, **i32)),
                dict(draft_prob=torch.zeros(3, 5, 100).bfloat16()), dict(draft_prob=torch.zeros(3, 5, 99)), dict(temperature=torch.zeros(3).double()),
                dict(tree_len=torch.zeros(3)), dict(logprob=torch.zeros(3, 5).double())):
        with pytest.raises(ValueError):
            kvq.tree_verify(**{**good, **bad})
    assert not calls
    kvq.tree_verify(**good)
    wide = torch.zeros(3, 7, 120).bfloat16()
    kvq.tree_verify(**{**good, "logits": wide[:, 1:6, 3:103], "tree_mask": torch.zeros(5, dtype=torch.int64), "draft_prob": torch.zeros(3, 6, 100)[:, :5]})
    assert calls[0][:3] == (3, 5, 100) and calls[0][4:7] == (1, 500, 100) and calls[0][9] == 5 and calls[0][10:13] == (0, 0, 0)
    assert calls[1][4:7] == (0, 840, 120) and calls[1][9] == 0 and calls[1][11:13] == (600, 100)


def test_binding_of_window(recorded):
    import numpy as np
    import torch
    L, calls = recorded
    q = torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16)
    good = dict(L=L, cache=FAKE, q=q, T=220, n_sink=4, window=64, out=torch.zeros_like(q))
    for bad in (dict(cache=torch.zeros(100, dtype=torch.uint8)), dict(q=q[0, 0]), dict(q=q.float()), dict(out=q[:, :2]), dict(lse=torch.zeros(2, 3, 7)),
                dict(seq_len=torch.zeros(2)), dict(T=2 ** 32 + 220), dict(n_sink=2 ** 31), dict(window=2 ** 33)):
        with pytest.raises(ValueError):
            kvq.decode_attention_window(**{**good, **bad})
    assert not calls
    kvq.decode_attention_window(**{**good, "T": np.int64(220), "lse": torch.zeros(2, 3, 8)})
    kvq.decode_attention_window(**{**good, "q": q[:, 0].contiguous(), "out": q[:, 0].contiguous(), "lse": torch.zeros(2, 8)})
    assert calls[0][3] == 3 and calls[0][5:8] == (220, 4, 64) and calls[1][3] == 1


def test_binding_refuses_another_device(lib):
    """CPU tensors with no stand-ins: the device is refused."""
    import torch
    L = _layout()
    q = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.decode_attention_window(L, FAKE, q, 220, 4, 64, q.clone(), stream=0)
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.norm_rope(L, _desc(), q, None, torch.zeros(3, 2, 1, dtype=torch.int32), torch.zeros(64), q.clone(), None, stream=0)
    x = torch.zeros(3, 5, 10)
    i = torch.zeros(3, 5, dtype=torch.int32)
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.tree_verify(x, i, torch.zeros(3, 5, dtype=torch.int64), x[..., 0], x[:, 0], i, i[:, 0], i[:, 0], stream=0)
