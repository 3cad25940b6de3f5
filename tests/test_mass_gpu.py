"""kvq_attention_mass against 64-bit references over the oracle's
reconstruction of the cache (tests/serving_ref.py has the tolerance)."""
import numpy as np
import pytest
import torch

import bit_mixed_precision_kvq_gb300 as kvq
import oracle
from gpu_helpers import Case, bits
from serving_ref import SCALE, Filled, bf16, check_mass, f64

pytestmark = pytest.mark.gpu


def _lse(c, q, khat, lens, taken):
    """lse of the taken tokens over what each reaches, fp32 [B, n_q, H_q] (0 elsewhere)."""
    out = np.zeros(q.shape[:3], np.float32)
    g = c.H_q // c.H_kv
    for b, toks in enumerate(taken):
        for k, tok in enumerate(toks if lens[b] is not None else []):
            end = lens[b] - len(toks) + 1 + k
            for hq in range(c.H_q):
                s = SCALE * (khat[b, hq // g, :end] @ q[b, tok, hq])
                out[b, tok, hq] = s.max() + np.log(np.exp(s - s.max()).sum()) if end > 0 else -np.inf
    return out


def _run(F, q, lse, T, decay, mass_in, lens=None, path=None, counts=None, in_place=False, dev="cuda"):
    c = F.c
    t = lambda x, d: None if x is None else torch.tensor(np.asarray(x), dtype=d, device=dev)  # noqa: E731
    mass = mass_in.clone() if in_place else torch.full((c.B, c.H_kv, c.T_cap), -3.0, device=dev)
    before = mass.clone()
    kvq.attention_mass(F.L, F.cache, q, torch.from_numpy(lse).to(dev), T, mass, mass if in_place else mass_in, SCALE, decay,
                       seq_len=t(lens, torch.int32), path=t(path, torch.int32), path_len=t(counts, torch.int32))
    torch.cuda.synchronize()
    return mass, before


CASES = [
    # layout, n_q, T, lengths
    (Case(1, 4, 1, 300, 14, 256, 4, 4, 32, []), 1, 257, None),
    (Case(1, 28, 4, 700, 14, 640, 4, 2, 64, [0]), 1, 690, None),
    (Case(2, 8, 8, 300, 10, 250, 8, 4, 32, [1], konly=[2]), 8, 300, None),
    (Case(2, 32, 8, 500, 32, 400, 2, 2, 32, [3]), 3, 480, None),
    (Case(1, 4, 4, 400, 16, 300, 2, 4, 128, [0]), 64, 400, None),
    (Case(3, 6, 2, 300, 0, 290, 16, 16, 64, [], konly=[1]), 7, 295, None),
    (Case(2, 5, 1, 300, 8, 8, 4, 4, 64, []), 9, 200, None),
    (Case(5, 8, 2, 300, 16, 272, 4, 2, 64, [1]), 3, 290, [3, 2, 0, 291, 200]),   # all causal, too short, empty, too long
    (Case(2, 16, 1, 700, 5, 650, 2, 8, 32, []), 12, 680, [128, 133]),            # 192 columns
    (Case(40, 4, 4, 200, 16, 144, 4, 2, 64, [2]), 1, 1, None),                   # one position
    (Case(1, 256, 2, 300, 3, 200, 8, 2, 64, []), 2, 210, None),                  # 256 columns per KV head
]


@pytest.mark.parametrize("ci", range(len(CASES)))
def test_mass_matches_reference(cuda_dev, kvq, ci):
    c, n_q, T, lens = CASES[ci]
    F = Filled(c, 5000 + 10 * ci, cuda_dev)
    q = bf16((c.B, n_q, c.H_q, c.D), 5003 + 10 * ci, cuda_dev)
    act = [n if 1 <= n <= T and n_q <= n else None for n in (lens or [T] * c.B)]
    taken = [list(range(n_q))] * c.B
    lse = _lse(c, f64(q), F.khat, act, taken)
    mass_in = torch.rand(c.B, c.H_kv, c.T_cap, device=cuda_dev)
    for decay, m_in, in_place in ((0.9, mass_in, False), (1.0, mass_in, True), (0.5, None, False)):
        got, before = _run(F, q, lse, T, decay, m_in, lens, in_place=in_place)
        check_mass(c, got, f64(q), lse, F.khat, act, taken, None if m_in is None else f64(m_in), decay, before)
    if n_q == 1:  # one query: the weights of each query head sum to 1
        for b in range(c.B):
            if act[b] is not None:
                s = f64(got)[b, :, :act[b]].sum(-1)
                assert np.abs(s - c.H_q // c.H_kv).max() <= 1e-4 * (c.H_q // c.H_kv)


@pytest.mark.parametrize("kb,G", [(kb, G) for kb in (2, 4, 8, 16) for G in (32, 64, 128)])
def test_mass_every_width(cuda_dev, kvq, kb, G):
    c = Case(1, 9, 3, 330, 13, 300, kb, 4, G, [1], konly=[2])
    F = Filled(c, 5300, cuda_dev)
    k = F.k.clone()
    k[..., [3, 40, 77, 126]] *= 10
    kvq.quantize_append(F.L, F.cache, k, F.v, 0)
    khat = oracle.reconstruct(bits(k), c.vs, c.ve, c.mask(), kb, G)[0]
    q = bf16((1, 5, 9, 128), 5303, cuda_dev)
    lse = _lse(c, f64(q), khat, [321], [range(5)])
    got, before = _run(F, q, lse, 321, 1.0, None)
    check_mass(c, got, f64(q), lse, khat, [321], [range(5)], None, 1.0, before)


def test_mass_along_a_path(cuda_dev, kvq):
    """Tokens picked by a path, in any order and twice, none, one past its
    range (adds nothing), and a path longer than the sequence (inactive)."""
    c = Case(6, 6, 2, 300, 10, 250, 4, 4, 64, [0])
    F = Filled(c, 5400, cuda_dev)
    n_q, T = 9, 280
    q = bf16((6, n_q, 6, 128), 5401, cuda_dev)
    path = [[0, 3, 7, -1], [8, 2, 2, 1], [-1] * 4, [4, 9, 5, 0], [0, 1, 2, 3], [1, 2, 3, 4]]
    counts, lens = [3, 4, 0, 3, 5, 4], [280, 260, 270, 255, 280, 3]
    act = [280, 260, 270, 255, None, None]
    taken = [[0, 3, 7], [8, 2, 2, 1], [], [4, 9, 5], [], []]
    lse = (np.random.default_rng(0).random((6, n_q, 6)).astype(np.float32) + 7.0)
    mass_in = torch.rand(6, 2, 300, device=cuda_dev)
    got, before = _run(F, q, lse, T, 0.75, mass_in, lens, path, counts)
    big = np.concatenate([lse, np.full((6, 1, 6), np.inf, np.float32)], 1)   # token 9 adds nothing
    q9 = np.concatenate([f64(q), np.zeros((6, 1, 6, 128))], 1)
    check_mass(c, got, q9, big, F.khat, act, taken, f64(mass_in), 0.75, before)


def test_mass_rows_without_weight(cuda_dev, kvq):
    """lse of -inf (a row that attended nothing) and +inf add nothing, also
    where their queries are NaN; NaN past the length is not looked at."""
    c = Case(2, 4, 2, 200, 6, 150, 8, 8, 64, [])
    F = Filled(c, 5500, cuda_dev)
    q = bf16((2, 3, 4, 128), 5501, cuda_dev)
    want = f64(q)
    lse = np.full((2, 3, 4), 6.0, np.float32)
    lse[0, 1], lse[1, 2, 0] = -np.inf, np.inf
    q[0, 1] = float("nan")
    late = torch.full((2, 2, 20, 128), float("nan"), dtype=torch.bfloat16, device=cuda_dev)
    kvq.quantize_append(F.L, F.cache, late, late, 180)
    mass_in = torch.rand(2, 2, 200, device=cuda_dev)
    mass_in[:, :, 180:] = float("nan")
    got, before = _run(F, q, lse, 180, 1.0, mass_in)
    check_mass(c, got, want, lse, F.khat, [180, 180], [range(3)] * 2, np.nan_to_num(f64(mass_in)), 1.0, before)


def test_mass_of_a_decode_call(cuda_dev, kvq):
    """With the lse that kvq_decode_attention returned: sums of 1 per query head."""
    c = Case(2, 28, 4, 1500, 14, 1400, 4, 2, 64, [0])
    F = Filled(c, 5600, cuda_dev)
    q = bf16((2, 28, 128), 5601, cuda_dev)
    out, lse = torch.empty_like(q), torch.empty(2, 28, device=cuda_dev)
    ws = torch.zeros(int(F.L.workspace_bytes), dtype=torch.uint8, device=cuda_dev)
    kvq.decode_attention(F.L, F.cache, q, 1450, out, SCALE, lse, ws)
    mass = torch.zeros(2, 4, 1500, device=cuda_dev)
    kvq.attention_mass(F.L, F.cache, q, lse, 1450, mass, None, SCALE)
    torch.cuda.synchronize()
    assert float((mass.double().sum(-1) - 7).abs().max()) <= 7 * 1e-4
    assert not mass[:, :, 1450:].any()


@pytest.mark.parametrize("kb,G", [(2, 32), (4, 64), (8, 128)])
def test_mass_long_runs_and_many_columns(cuda_dev, kvq, kb, G):
    """Several blocks a warp and two passes over them (96 columns), in place,
    with lengths that end in the prefix, inside a block and behind the visual
    rows."""
    c = Case(80, 32, 2, 700, 9, 650, kb, 2, G, [])
    F = Filled(c, 5700, cuda_dev)
    n_q, T = 6, 690
    q = bf16((80, n_q, 32, 128), 5701, cuda_dev)
    lens = [T - (7 * b) % 400 for b in range(80)]
    lens[3], lens[4] = 8, 650
    lse = _lse(c, f64(q), F.khat, lens, [list(range(n_q))] * 80)
    mass_in = torch.rand(80, 2, 700, device=cuda_dev)
    got, before = _run(F, q, lse, T, 0.9, mass_in, lens, in_place=True)
    check_mass(c, got, f64(q), lse, F.khat, lens, [list(range(n_q))] * 80, f64(mass_in), 0.9, before)
