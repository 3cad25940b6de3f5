"""Refusals of the tree, commit, mass and eviction calls: every case is
rejected on the host before any CUDA call (the addresses are never
dereferenced), and the Python binding's own checks."""
import ctypes

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


def test_tree_workspace_bytes(lib):
    L = _layout()
    assert kvq.decode_tree_workspace_bytes(L, 1) >= 256
    assert kvq.decode_tree_workspace_bytes(L, 64) >= kvq.decode_tree_workspace_bytes(L, 1)
    for n_q in (0, -1, 65):
        assert kvq.decode_tree_workspace_bytes(L, n_q) == 0
    bad = kvq.Layout.from_buffer_copy(L)
    bad.n_packed += 1
    assert kvq.decode_tree_workspace_bytes(bad, 4) == 0


TREE_BAD = [
    (dict(cache=0), 1), (dict(cache=FAKE + 128), 1), (dict(q=0), 1), (dict(q=FAR + 8), 1), (dict(kd=0), 1),
    (dict(vd=0), 1), (dict(kd=2 * FAR + 8), 1), (dict(vd=FAKE), 1),            # a draft inside the cache
    (dict(kd=FAKE - 256), 1),                                                  # ... reaching into it
    (dict(sb=-8), 1), (dict(sh=4), 1), (dict(st=12), 1), (dict(sb=1 << 60), 1), (dict(n_q=0), 1), (dict(n_q=65), 1),
    (dict(mask=0), 1), (dict(mask=FAR + 4), 1), (dict(msb=3), 1), (dict(msb=-4), 1), (dict(seq=FAR + 2), 1),
    (dict(T=-1), 1), (dict(T=257), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(out=0), 1), (dict(out=FAR + 2), 1), (dict(lse=FAR + 1), 1), (dict(ws=0), 1), (dict(ws=FAR + 16), 1),
    (dict(wsb=-1), 3),
]


@pytest.mark.parametrize("bad,code", TREE_BAD, ids=lambda x: str(x)[:40])
def test_tree_argument_checks(lib, bad, code):
    L = _layout()
    a = dict(cache=FAKE, q=FAR, kd=2 * FAR, vd=3 * FAR, sb=4 * 4 * 128, sh=4 * 128, st=128, n_q=4, mask=4 * FAR, msb=4,
             seq=0, T=220, scale=0.1, out=5 * FAR, lse=0, ws=6 * FAR, wsb=0)
    a.update(bad)
    need = kvq.decode_tree_workspace_bytes(L, a["n_q"]) + a["wsb"]
    st = lib.kvq_decode_attention_tree(ctypes.byref(L), a["cache"], a["q"], a["kd"], a["vd"], a["sb"], a["sh"], a["st"],
                                       a["n_q"], a["mask"], a["msb"], a["seq"], a["T"], a["scale"], a["out"], a["lse"],
                                       a["ws"], max(0, need), None)
    assert st == code


COMMIT_BAD = [
    dict(cache=0), dict(cache=FAKE + 64), dict(kd=0), dict(vd=0), dict(kd=FAKE + 256), dict(sb=-8), dict(sh=4),
    dict(st=1), dict(n_q=0), dict(n_q=65), dict(path=0), dict(path=FAR + 2), dict(plen=0), dict(plen=FAR + 2),
    dict(maxp=0), dict(maxp=65), dict(seq=FAR + 1), dict(T=-1), dict(T=257), dict(new=FAR + 2),
    dict(new=7 * FAR, seq=7 * FAR),           # the new lengths in place of the old
    dict(new=7 * FAR + 4, seq=7 * FAR),       # ... one entry apart
    dict(new=5 * FAR), dict(new=4 * FAR + 12),  # ... over the path lengths, over the path
]


@pytest.mark.parametrize("bad", COMMIT_BAD, ids=lambda x: str(x)[:40])
def test_commit_argument_checks(lib, bad):
    L = _layout()
    a = dict(cache=FAKE, kd=2 * FAR, vd=3 * FAR, sb=4 * 4 * 128, sh=4 * 128, st=128, n_q=4, path=4 * FAR, maxp=3,
             plen=5 * FAR, seq=0, T=220, new=0)
    a.update(bad)
    st = lib.kvq_tree_commit(ctypes.byref(L), a["cache"], a["kd"], a["vd"], a["sb"], a["sh"], a["st"], a["n_q"], a["path"],
                             a["maxp"], a["plen"], a["seq"], a["T"], a["new"], None)
    assert st == 1


MASS_BAD = [
    dict(cache=0), dict(cache=FAKE + 8), dict(q=0), dict(q=FAR + 2), dict(lse=0), dict(lse=FAR + 2), dict(n_q=0),
    dict(n_q=65), dict(T=0), dict(T=257), dict(n_q=5, T=4), dict(seq=FAR + 2), dict(path=FAR), dict(plen=FAR),
    dict(path=FAR, plen=2 * FAR, maxp=0), dict(path=FAR, plen=2 * FAR, maxp=65), dict(path=FAR + 2, plen=2 * FAR, maxp=4),
    dict(path=FAR, plen=2 * FAR + 2, maxp=4), dict(scale=float("inf")), dict(decay=float("nan")), dict(mass=0),
    dict(mass=5 * FAR + 2), dict(mass_in=5 * FAR + 4), dict(mass_in=6 * FAR + 1),
]


@pytest.mark.parametrize("bad", MASS_BAD, ids=lambda x: str(x)[:40])
def test_mass_argument_checks(lib, bad):
    L = _layout()
    a = dict(cache=FAKE, q=FAR, lse=2 * FAR, n_q=4, seq=0, T=220, path=0, maxp=0, plen=0, scale=0.1, mass_in=0, decay=1.0,
             mass=5 * FAR)
    a.update(bad)
    st = lib.kvq_attention_mass(ctypes.byref(L), a["cache"], a["q"], a["lse"], a["n_q"], a["seq"], a["T"], a["path"],
                                a["maxp"], a["plen"], a["scale"], a["mass_in"], a["decay"], a["mass"], None)
    assert st == 1


def _evict(lib, L, D, **bad):
    a = dict(cache=FAKE, mass=FAR, seq=0, T=220, dst=2 * FAR, T_dst=120, recent=4, keep=3 * FAR, mass_dst=0, new=0)
    a.update(bad)
    return lib.kvq_cache_evict(ctypes.byref(L), a["cache"], a["mass"], a["seq"], a["T"], ctypes.byref(D), a["dst"],
                               a["T_dst"], a["recent"], a["keep"], a["mass_dst"], a["new"], None)


EVICT_BAD = [
    (dict(cache=0), 1), (dict(cache=FAKE + 8), 1), (dict(dst=0), 1), (dict(dst=2 * FAR + 8), 1), (dict(dst=FAKE), 1),
    (dict(dst=FAKE + 256), 1), (dict(mass=0), 1), (dict(mass=FAR + 2), 1), (dict(keep=0), 1), (dict(keep=FAR + 3), 1),
    (dict(T=199), 1), (dict(T=257), 1), (dict(T_dst=109), 1), (dict(T_dst=151), 3), (dict(recent=-1), 1),
    (dict(recent=11), 1), (dict(mass_dst=FAR + 2), 1), (dict(mass_dst=FAR), 1), (dict(mass_dst=FAR + 4096), 1),
    (dict(seq=FAR + 1), 1), (dict(new=FAR + 2), 1), (dict(new=4 * FAR, seq=4 * FAR), 1),
]


@pytest.mark.parametrize("bad,code", EVICT_BAD, ids=lambda x: str(x)[:40])
def test_evict_argument_checks(lib, bad, code):
    assert _evict(lib, _layout(), _layout(T_cap=150, vis_end=110), **bad) == code


@pytest.mark.parametrize("other", [dict(B=1), dict(H_q=4), dict(H_kv=8, H_q=8), dict(vis_start=9), dict(vis_end=201),
                                   dict(k_bits=2), dict(v_bits=8), dict(group_size=64), dict(protected=[2]),
                                   dict(protected=[], k_only=[1])], ids=str)
def test_evict_refuses_another_kind_of_cache(lib, other):
    a = dict(T_cap=256, vis_end=110)
    a.update(other)
    assert _evict(lib, _layout(), _layout(**a), T_dst=a["vis_end"] + 10) == 1


def test_corrupted_layouts_are_refused(lib):
    L, D = _layout(), _layout(T_cap=150, vis_end=110)
    bad = kvq.Layout.from_buffer_copy(L)
    bad.off[2] += 256
    worse = kvq.Layout.from_buffer_copy(D)
    worse.Tv += 1
    assert _evict(lib, bad, D) == 1 and _evict(lib, L, worse) == 1
    assert lib.kvq_attention_mass(ctypes.byref(bad), FAKE, FAR, FAR, 1, None, 10, None, 0, None, 0.1, None, 1.0, 5 * FAR,
                                  None) == 1
    assert lib.kvq_tree_commit(ctypes.byref(bad), FAKE, FAR, 2 * FAR, 512, 128, 128, 1, 3 * FAR, 1, 4 * FAR, None, 10, None,
                               None) == 1
    assert lib.kvq_decode_attention_tree(ctypes.byref(bad), FAKE, FAR, 2 * FAR, 3 * FAR, 512, 128, 128, 1, 4 * FAR, 0, None,
                                         10, 0.1, 5 * FAR, None, 6 * FAR, 1 << 40, None) == 1


def test_binding_refuses_other_types_and_shapes(lib):
    """The binding checks what the C call cannot see (CPU tensors here: the
    device is refused too)."""
    import torch
    L = _layout()
    cache = torch.zeros(int(L.total_bytes), dtype=torch.uint8)
    q = torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16)
    kd = torch.zeros(2, 4, 3, 128, dtype=torch.bfloat16)
    mask = torch.zeros(2, 3, dtype=torch.int64)
    out, ws = torch.zeros_like(q), torch.zeros(256, dtype=torch.uint8)

    def tree(**kw):
        a = dict(cache=FAKE, q=q, k_draft=kd, v_draft=kd, tree_mask=mask, T_ctx=220, out=out, workspace=ws)
        a.update(kw)
        with pytest.raises(ValueError) as e:
            kvq.decode_attention_tree(L, a["cache"], a["q"], a["k_draft"], a["v_draft"], a["tree_mask"], a["T_ctx"], a["out"],
                                      workspace=a["workspace"], lse=kw.get("lse"), seq_len=kw.get("seq_len"), stream=0)
        return str(e.value)

    assert "current CUDA device" in tree()
    assert "cache" in tree(cache=cache[:100])
    assert "q" in tree(q=q[0])
    assert "bfloat16" in tree(q=q.float())
    mass = torch.zeros(2, 4, 256)
    for kw in (dict(q=q[0]), dict(q=q.half()), dict(lse=torch.zeros(2, 3, 7)), dict(mass=torch.zeros(2, 4, 255)),
               dict(mass_in=mass.double()), dict(path=torch.zeros(2, 2)), dict(path=torch.zeros(2, dtype=torch.int32))):
        a = dict(q=q, lse=torch.zeros(2, 3, 8), mass=mass, mass_in=None, path=None)
        a.update(kw)
        with pytest.raises(ValueError):
            kvq.attention_mass(L, FAKE, a["q"], a["lse"], 220, a["mass"], a["mass_in"], path=a["path"],
                               path_len=a["path"], stream=0)
    with pytest.raises(ValueError):
        kvq.tree_commit(L, FAKE, kd, kd.transpose(1, 2), torch.zeros(2, 2, dtype=torch.int32),
                        torch.zeros(2, dtype=torch.int32), 220, stream=0)
    with pytest.raises(ValueError):
        kvq.cache_evict(L, FAKE, mass, 220, L, FAKE, 210, torch.zeros(2, 4, 209, dtype=torch.int32), stream=0)
