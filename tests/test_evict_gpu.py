"""kvq_cache_evict: the kept positions, masses and lengths equal the
reference's, and every kept row is copied bit for bit."""
import numpy as np
import pytest
import torch

import bit_mixed_precision_kvq_gb300 as kvq
from gpu_helpers import Case
from serving_ref import Filled, keep_reference

pytestmark = pytest.mark.gpu


def _segment(L, cache, seg, heads, rows):
    o, w = int(L.off[seg]), int(L.row_bytes[seg])
    n = int(L.d.B) * heads * rows
    return cache[o:o + n * w].view(int(L.d.B), heads, rows, w) if w and n else None


def _rows_of(c, L, cache):
    """(segment, KV heads, stored rows, visual) of the eight segments."""
    prot, konly = list(c.prot), list(c.konly)
    pack = [h for h in range(c.H_kv) if h not in prot + konly]
    every = list(range(c.H_kv))
    heads = [pack, pack, pack + konly, pack + konly, prot + konly, prot, every, every]
    rows = [int(L.Tv_pad)] * 4 + [int(L.Tv)] * 2 + [int(L.T_text)] * 2
    return [(h, _segment(L, cache, s, len(h), rows[s]), s < 6) for s, h in enumerate(heads)]


def _evict(F, mass, T, k_vis, k_text, recent, lens=None, spare=9, optional=True, dev="cuda"):
    c = F.c
    D = Case(c.B, c.H_q, c.H_kv, c.vs + k_vis + k_text + spare, c.vs, c.vs + k_vis, c.kb, c.vb, c.G, c.prot, konly=c.konly)
    Ld = D.layout()
    T_dst = c.vs + k_vis + k_text
    dst = torch.full((int(Ld.total_bytes),), 0x5A, dtype=torch.uint8, device=dev)
    keep = torch.full((c.B, c.H_kv, T_dst), 12345, dtype=torch.int32, device=dev)
    mass_dst = torch.full((c.B, c.H_kv, D.T_cap), -5.0, device=dev) if optional else None
    new = torch.full((c.B,), 77, dtype=torch.int32, device=dev) if optional else None
    sl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
    kvq.cache_evict(F.L, F.cache, mass, T, Ld, dst, T_dst, keep, recent, mass_dst, sl, new)
    torch.cuda.synchronize()
    act = [n if c.ve <= n <= T else None for n in (lens or [T] * c.B)]
    want = keep_reference(c, mass.cpu().numpy(), act, k_vis, k_text, recent)
    got = keep.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:4]
    ends = [c.vs + k_vis + min(k_text, n - c.ve) if n is not None else -1 for n in act]
    if optional:
        assert new.tolist() == ends
        for b, n in enumerate(ends):
            x = mass_dst[b]
            if n < 0:
                assert (x == -5.0).all()
                continue
            at = torch.from_numpy(want[b, :, :n]).to(dev)
            assert torch.equal(x[:, :n].view(torch.int32), mass[b].gather(1, at).view(torch.int32)) and not x[:, n:].any()
    src, out = _rows_of(c, F.L, F.cache), _rows_of(c, Ld, dst)
    touched = torch.zeros_like(dst, dtype=torch.bool)
    for (heads, a, visual), (_, y, _), (_, seen, _) in zip(src, out, _rows_of(c, Ld, touched.view(torch.uint8))):
        if a is None or y is None:
            continue
        for b, n in enumerate(ends):
            for i, h in enumerate(heads if n >= 0 else []):
                if visual:
                    at = want[b, h, c.vs:c.vs + k_vis] - c.vs
                else:
                    t = np.concatenate([want[b, h, :c.vs], want[b, h, c.vs + k_vis:n]])
                    at = np.where(t >= c.ve, t - (c.ve - c.vs), t)
                at = torch.from_numpy(at).to(dev)
                assert torch.equal(y[b, i, :len(at)], a[b, i].index_select(0, at)), (heads, b, h)
                seen[b, i, :len(at)] = 1
    assert (dst[~touched.view(torch.bool)] == 0x5A).all()   # nothing else is written


def _mass(c, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    m = torch.randn(c.B, c.H_kv, c.T_cap, device=dev, generator=g).mul_(2).exp_()
    return m * (torch.rand(m.shape, device=dev, generator=g) > 0.2)   # ties at exactly 0


CASES = [
    # layout, T, kept visual, kept text, recent, lengths
    (Case(1, 4, 1, 300, 14, 256, 4, 4, 32, []), 280, 100, 10, 3, None),
    (Case(1, 28, 4, 1700, 14, 1640, 4, 2, 64, [0]), 1690, 820, 50, 16, None),     # all 50 text rows stay
    (Case(2, 8, 8, 300, 10, 250, 8, 4, 32, [1], konly=[2]), 300, 239, 20, 20, None),  # only recent text
    (Case(2, 8, 8, 300, 10, 250, 8, 4, 32, [1], konly=[2]), 299, 240, 0, 0, None),    # all visual rows, no text
    (Case(2, 32, 8, 500, 32, 400, 2, 2, 128, [3]), 480, 0, 30, 0, None),          # no visual row stays
    (Case(3, 6, 2, 300, 0, 290, 16, 16, 64, [], konly=[1]), 295, 17, 5, 2, None),
    (Case(2, 5, 1, 300, 8, 8, 4, 4, 64, []), 200, 0, 100, 10, None),              # no visual block
    (Case(2, 5, 1, 300, 0, 0, 4, 4, 64, []), 200, 0, 1, 1, None),                 # one row
    (Case(7, 8, 2, 300, 16, 200, 4, 2, 64, [1]), 290, 33, 40, 5, [200, 201, 205, 240, 241, 199, 291]),
    (Case(2, 8, 2, 9000, 3, 8900, 2, 2, 32, []), 8950, 1, 7, 7, None),
    (Case(1, 4, 2, 40000, 30, 39000, 2, 4, 64, []), 39500, 20001, 250, 100, None),
]


@pytest.mark.parametrize("ci", range(len(CASES)))
def test_evict_matches_reference(cuda_dev, kvq, ci):
    c, T, k_vis, k_text, recent, lens = CASES[ci]
    F = Filled(c, 6000 + 10 * ci, cuda_dev) if c.T_cap < 20000 else _quick(c, cuda_dev)
    _evict(F, _mass(c, 6001 + ci, cuda_dev), T, k_vis, k_text, recent, lens)


class _quick:
    """A cache of random bytes: eviction does not look into rows."""

    def __init__(self, c, dev):
        self.c, self.L = c, c.layout()
        self.cache = torch.randint(0, 256, (int(self.L.total_bytes),), dtype=torch.uint8, device=dev)


@pytest.mark.parametrize("kb,vb,G", [(2, 16, 32), (4, 8, 128), (8, 2, 64), (16, 4, 32), (2, 2, 128)])
def test_evict_every_row_size(cuda_dev, kvq, kb, vb, G):
    c = Case(2, 6, 3, 400, 5, 333, kb, vb, G, [0], konly=[2])
    _evict(_quick(c, cuda_dev), _mass(c, 6200, cuda_dev), 371, 101, 13, 4)


def test_evict_values_that_tie(cuda_dev, kvq):
    """Equal masses, signed zeros, infinities, NaN, subnormals and negative
    values: NaN last, ties to the lowest position."""
    c = Case(2, 4, 2, 700, 6, 600, 4, 4, 64, [])
    F = _quick(c, cuda_dev)
    g = torch.Generator(device=cuda_dev).manual_seed(1)
    few = torch.tensor([0.0, -0.0, 1.0, -1.0, float("inf"), -float("inf"), float("nan"), 1e-42, -1e-42, 3.0], device=cuda_dev)
    mass = few[torch.randint(0, 10, (2, 2, 700), device=cuda_dev, generator=g)]
    for k_vis, k_text, recent in ((1, 1, 0), (59, 10, 3), (300, 50, 0), (593, 79, 0), (594, 80, 80)):
        _evict(F, mass, 680, k_vis, k_text, recent)
    for same in (0.0, 2.5, float("nan")):
        _evict(F, torch.full_like(mass, same), 680, 123, 45, 6, [680, 650])


def test_evict_without_optional_outputs(cuda_dev, kvq):
    c = Case(2, 4, 2, 300, 14, 256, 4, 4, 32, [])
    _evict(_quick(c, cuda_dev), _mass(c, 6300, cuda_dev), 280, 100, 10, 3, spare=0, optional=False)


# Ranges on both sides of what the registers of each size of CTA hold:
# (B, KV heads, visual, text, lengths)
LONG = [(1, 1, 1024, 40, None), (1, 1, 4096, 40, None), (1, 1, 8192, 4, None), (1, 1, 8193, 4, None), (1, 1, 1025, 40, None), (3, 2, 1060, 1500, [2600, 1065, 1064]), (1, 2, 4097, 5, None),
        (1, 1, 32768, 3, None), (2, 1, 32769, 40, None), (1, 1, 70001, 33000, None), (2, 80, 1111, 60, None),
        (2, 1, 0, 9001, [9005, 20])]


@pytest.mark.parametrize("case", LONG)
def test_evict_long_ranges(cuda_dev, kvq, case):
    """Random masses, masses of three values (the last kept one's equals are
    spread over the whole range) and equal ones."""
    B, H, n_vis, n_text, lens = case
    vs = 5
    c = Case(B, H, H, vs + n_vis + n_text + 11, vs, vs + n_vis, 2, 2, 128, [])
    F = _quick(c, cuda_dev)
    T = vs + n_vis + n_text
    m = _mass(c, 6400, cuda_dev)
    three = m.clamp(max=1.0).mul(2).round()
    for mass in (m, three, torch.ones_like(m)):
        _evict(F, mass, T, n_vis // 3, max(n_text // 2, 1), min(3, n_text // 2), lens)
    _evict(F, three, T, n_vis, n_text, 0, lens)
