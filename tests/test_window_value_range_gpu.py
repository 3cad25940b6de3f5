"""kvq_decode_attention_window with finite bf16 V rows of any size, to the largest:
text rows, heads that keep bf16 rows, 16-bit caches, beside packed rows."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import Case, append, bits
from serving_ref import Filled, bf16, f64, score_error
from step_ref import window_reference

pytestmark = pytest.mark.gpu
MOST = 2.0 ** 128 - 2.0 ** 120  # the largest finite bf16


def with_values(c, F, v):
    """F's cache with the V rows v, and the values that they stand for."""
    append(F.L, F.cache, F.k, v, 0)
    m = [1 if x == 1 else 0 for x in c.mask()]
    return oracle.reconstruct(bits(v), c.vs, c.ve, m, c.vb, c.G)[0]


def check(c, out, lse, q, khat, vhat, lens, n_sink, window):
    """One bf16 rounding (2^-8 of the value; 2^-133 below bf16's normal range).
    Against the largest |v| of the element over the positions: a score's error e
    moves a weight by a factor of e^(2e); bf16 rows' weights are off by 2^-17, packed
    ones' by 2^-11, and by 2^-11 again of code * scale <= 2 max|V| where they meet it;
    what those lose below fp16's normal range is 2^-28 for a position (check_window)."""
    ref, lr = window_reference(c, q, khat, vhat, lens, n_sink, window)
    g = c.H_q // c.H_kv
    se = score_error(q, khat)[..., None]
    vd = np.repeat(np.abs(vhat).max(axis=2), g, axis=1)[:, None]                # [B, 1, H_q, D]
    kept = np.repeat(np.array([m == 1 or c.vb == 16 for m in c.mask()]), g)[None, None, :, None]
    rows = min(khat.shape[2], n_sink + window + q.shape[1])
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -133 + np.where(kept, 2.0 ** -16 + 2 * se, 3 * 2.0 ** -11 + 2 * se) * vd + np.where(kept, 0, rows * 2.0 ** -28 * np.maximum(1, vd))
    o = f64(out)
    assert np.all(np.isfinite(o))
    err = np.abs(o - ref)
    assert np.all(err <= tol), f"out: worst err / tol {np.max(err / tol):.3g}"
    l = f64(lse)
    le, lt = np.abs(l - lr), se[..., 0] + 2.0 ** -21 * (1 + np.abs(lr))
    assert np.all(le <= lt), f"lse: worst err / tol {np.max(le / lt):.3g}"


def run(kvq, dev, f, q, T, n_sink, window, lens=None):
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device=dev)
    kvq.decode_attention_window(f.L, f.cache, q, T, n_sink, window, out, None, lse,
                                None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev))
    return out, lse


def sized(c, v, kind, size):
    """Rows of v with bf16 rows of size `size`; packed rows stay ordinary."""
    v = v.clone()
    keeps = [h for h in range(c.H_kv) if c.mask()[h] == 1 or c.vb == 16]
    t = torch.arange(c.T_cap, device=v.device)
    text = (t < c.vs) | (t >= c.ve)
    big = torch.zeros(1, c.H_kv, c.T_cap, 1, dtype=torch.bool, device=v.device)
    big[:, :, text] = True
    big[:, keeps] = True
    unit = (v.float() / v.float().abs().max()).clamp(-1, 1)
    if kind == "one sign":      # every element the size itself: sums of it must not overflow either
        unit = torch.ones_like(unit)
    elif kind == "some elements":
        big = big & (torch.arange(128, device=v.device) % 7 == 3)
    elif kind == "one row":
        big = big & (t == (c.ve + 3 if c.ve < c.T_cap - 20 else 5))[:, None]
    elif kind == "beside tiny":  # ordinary ones become tiny in the heads that keep bf16 rows
        small = torch.zeros_like(big)
        small[:, keeps] = True
        v = torch.where(small, (v.float() * 2.0 ** -60).bfloat16(), v)
        big = big & (torch.arange(128, device=v.device) < 40)
    return torch.where(big, (unit.double() * size).to(torch.bfloat16), v)


KINDS = ["all", "one sign", "some elements", "one row", "beside tiny"]


@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** 113, 2.0 ** 117, MOST])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("vb", [2, 8, 16])
def test_values_to_the_largest(cuda_dev, kvq, vb, kind, size):
    c = Case(1, 4, 2, 300, 10, 250, 4, vb, 32, [1])
    F = Filled(c, 16, cuda_dev)
    vhat = with_values(c, F, sized(c, F.v, kind, size))
    for n_q in (1, 2, 6):  # one and two tiles of columns
        q = bf16((1, n_q, 4, 128), 17 + n_q, cuda_dev)
        for n_sink, window in ((12, 270), (40, 100), (0, 300)):
            out, lse = run(kvq, cuda_dev, F, q, 299, n_sink, window)
            check(c, out, lse, f64(q), F.khat, vhat, [299], n_sink, window)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kb,vb,G", [(8, 4, 64), (2, 2, 128), (16, 8, 32), (16, 16, 32)])
def test_values_of_many_units(cuda_dev, kvq, kind, kb, vb, G):
    """One CTA a unit, K-only protected heads, lengths of their own."""
    c = Case(40, 32, 16, 180, 8, 160, kb, vb, G, [3, 7], konly=[5])
    F = Filled(c, 22, cuda_dev)
    vhat = with_values(c, F, sized(c, F.v, kind, MOST))
    q = bf16((40, 1, 32, 128), 23, cuda_dev)
    lens = [175 - b % 11 for b in range(40)]
    out, lse = run(kvq, cuda_dev, F, q, 175, 6, 90, lens)
    check(c, out, lse, f64(q), F.khat, vhat, lens, 6, 90)


@pytest.mark.parametrize("vb", [2, 16])
def test_values_of_a_long_window(cuda_dev, kvq, vb):
    """A unit of many CTAs, thousands of the largest rows."""
    c = Case(1, 14, 2, 9000, 14, 6000, 4, vb, 64, [0])
    F = Filled(c, 24, cuda_dev)
    for kind in ("all", "one sign", "one row"):
        vhat = with_values(c, F, sized(c, F.v, kind, MOST))
        q = bf16((1, 2, 14, 128), 25, cuda_dev)
        out, lse = run(kvq, cuda_dev, F, q, 8990, 30, 8000)
        check(c, out, lse, f64(q), F.khat, vhat, [8990], 30, 8000)


def test_faint_huge_rows_leave_the_others(cuda_dev, kvq):
    """Huge text rows whose weights are some 2^-60 of the others' beside packed
    rows: what they add is of the ordinary rows' size."""
    c = Case(1, 2, 1, 200, 8, 150, 16, 4, 32, [])
    F = Filled(c, 26, cuda_dev)
    k = F.k.clone()
    k[..., :4] = 0
    k[:, :, :8, 0] = -30.0
    k[:, :, 150:, 0] = -30.0
    v = sized(c, F.v, "all", 2.0 ** 60)
    append(F.L, F.cache, k, v, 0)
    khat = oracle.reconstruct(bits(k), c.vs, c.ve, c.mask(), c.kb, c.G)[0]
    vhat = oracle.reconstruct(bits(v), c.vs, c.ve, [0], c.vb, c.G)[0]
    q = (bf16((1, 1, 2, 128), 27, cuda_dev).float() * 0.05).bfloat16()
    q[..., 0] = 16.0  # -480 / sqrt(128) = -42.4: e^-42.4 = 2^-61
    out, lse = run(kvq, cuda_dev, F, q, 199, 8, 190)
    ref, lr = window_reference(c, f64(q), khat, vhat, [199], 8, 190)
    # scores are exact to 2^-19 * 3 * 30 * 16 / 11.3 = 2^-12: weights to 2^-11; values as in `check`
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 3 * 2.0 ** -11) * (np.abs(vhat[:, :, 8:150]).max() + 200 * 2.0 ** 60 * 2.0 ** -60)
    assert np.all(np.abs(f64(out) - ref) <= tol) and np.all(np.abs(f64(lse) - lr) < 2.0 ** -11)
