"""The serving calls away from unit scale: small queries against large keys,
large against small, columns of very different size in one call, and small
values."""
import numpy as np
import pytest
import torch

import bit_mixed_precision_kvq_gb300 as kvq
import oracle
from gpu_helpers import Case, bits
from serving_ref import SCALE, Filled, bf16, f64, masks_to, random_tree, score_error, tree_reference

pytestmark = pytest.mark.gpu


def _tree(F, q, kd, vd, masks, T, dev):
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full(q.shape[:3], 9.0, device=dev)
    ws = torch.zeros(kvq.decode_tree_workspace_bytes(F.L, q.shape[1]), dtype=torch.uint8, device=dev)
    kvq.decode_attention_tree(F.L, F.cache, q, kd, vd, masks_to(dev, masks), T, out, SCALE, lse, ws)
    torch.cuda.synchronize()
    assert kvq.workspace_status(ws) == 0
    return out, lse


def _scaled(c, seed, dev, n_q, qs, ks, vs):
    """A cache, drafts and queries of the given sizes (qs: one per token),
    below 6e4 in size, and what the cache stands for."""
    F = Filled(c, seed, dev)
    clip = lambda x, s: (x.float() * s).clamp(-6e4, 6e4).to(torch.bfloat16)  # noqa: E731
    k, v = clip(F.k, ks), clip(F.v, vs)
    kvq.quantize_append(F.L, F.cache, k, v, 0)
    khat = oracle.reconstruct(bits(k), c.vs, c.ve, c.mask(), c.kb, c.G)[0]
    vhat = oracle.reconstruct(bits(v), c.vs, c.ve, [1 if x == 1 else 0 for x in c.mask()], c.vb, c.G)[0]
    x = bf16((2, c.B, n_q, c.H_kv, 128), seed + 2, dev)
    kd, vd = clip(x[0], ks).transpose(1, 2), clip(x[1], vs).transpose(1, 2)
    per_token = torch.tensor([qs[i % len(qs)] for i in range(n_q)], device=dev)[:, None, None]
    q = clip(bf16((c.B, n_q, c.H_q, 128), seed + 3, dev), per_token)
    return F, khat, vhat, q, kd, vd


# sizes of the queries (in turn over the tokens) and of the keys
SIZES = [([5e-4], 2e4), ([1e-3], 1e3), ([1e-2], 1e2), ([1e2], 0.1), ([1.0, 1e-6, 5e-4, 1e2, 0.0], 1e2),
         ([3e-9, 1e-30, 3e-3], 1e4)]


def _check_scores(c, seed, dev, qs, ks):
    """lse and output within the bounds of unit scale, plus what K's smallest
    step in the operands (an element of K is off by 2^-23 at most, its zero
    point included) makes of a score."""
    n_q, T = 6, 321
    F, khat, vhat, q, kd, vd = _scaled(c, seed, dev, n_q, qs, ks, 1.0)
    masks = random_tree(n_q, 1, 5)
    out, lse = _tree(F, q, kd, vd, masks, T, dev)
    qf, kdf, vdf = f64(q), f64(kd), f64(vd)
    ref, lr = tree_reference(c, qf, khat, vhat, kdf, vdf, masks, [T])
    se = score_error(qf, khat, kdf) + 2.0 ** -23 * SCALE * np.abs(qf).sum(-1)
    le = np.abs(f64(lse) - lr) / (se + 2.0 ** -22 * (1 + np.abs(lr)))
    assert le.max() <= 1, f"lse: worst err / tol {le.max():.3g}"
    vmax = np.repeat(np.maximum(np.abs(vhat).max(axis=(2, 3)), np.abs(vdf).max(axis=(2, 3))), 3, axis=1)[:, None, :, None]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 330 * 2.0 ** -28 + 2 * se[..., None]) * vmax
    oe = np.abs(f64(out) - ref) / tol
    assert oe.max() <= 1, f"out: worst err / tol {oe.max():.3g}"


@pytest.mark.parametrize("kb", [2, 4, 8, 16])
@pytest.mark.parametrize("si", range(len(SIZES)))
def test_tree_scores_of_any_size(cuda_dev, kvq, si, kb):
    _check_scores(Case(1, 9, 3, 330, 13, 300, kb, 4, 32, [1], konly=[2]), 8000 + 10 * si, cuda_dev, *SIZES[si])


@pytest.mark.parametrize("kb,G", [(kb, G) for kb in (2, 4, 8, 16) for G in (32, 64, 128)])
def test_tree_small_keys(cuda_dev, kvq, kb, G):
    """Scales below fp16's normal numbers."""
    for ks in (1e-3, 2e-2):
        _check_scores(Case(1, 9, 3, 330, 13, 300, kb, 4, G, [1], konly=[2]), 8100, cuda_dev, [10.0 / ks], ks)


@pytest.mark.parametrize("vs", [1e-6, 1e-3, 1.0, 2e4])
@pytest.mark.parametrize("vb", [2, 4, 8, 16])
def test_tree_values_of_any_size(cuda_dev, kvq, vb, vs):
    """Values are rounded to 2^-11 of themselves or, below 2^-14, to steps of
    2^-24; a weighted mean of them is off by no more than one of them, plus
    the weights' own 2^-11."""
    c = Case(1, 9, 3, 330, 13, 300, 4, vb, 32, [1], konly=[2])
    n_q, T = 6, 321
    F, khat, vhat, q, kd, vd = _scaled(c, 8200, cuda_dev, n_q, [1.0], 1.0, vs)
    masks = random_tree(n_q, 1, 5)
    out, lse = _tree(F, q, kd, vd, masks, T, cuda_dev)
    qf, kdf, vdf = f64(q), f64(kd), f64(vd)
    ref, lr = tree_reference(c, qf, khat, vhat, kdf, vdf, masks, [T])
    se = score_error(qf, khat, kdf)[..., None]
    vmax = np.repeat(np.maximum(np.abs(vhat).max(axis=(2, 3)), np.abs(vdf).max(axis=(2, 3))), 3, axis=1)[:, None, :, None]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 330 * 2.0 ** -28 + 2 * se) * vmax + 2.0 ** -24
    oe = np.abs(f64(out) - ref) / tol
    assert oe.max() <= 1, f"out: worst err / tol {oe.max():.3g}"


@pytest.mark.parametrize("T", [90, 2300])   # one CTA per unit, and units split over several
def test_tree_query_that_is_not_finite(cuda_dev, kvq, T):
    """NaN in a token's query: NaN in that token's rows and lse, nowhere else."""
    c = Case(1, 8, 2, 2400, 10, 2200, 4, 4, 64, [1])
    F = Filled(c, 8300, cuda_dev)
    n_q = 5
    q, x = bf16((1, n_q, 8, 128), 8301, cuda_dev), bf16((2, 1, n_q, 2, 128), 8302, cuda_dev)
    kd, vd = x[0].transpose(1, 2), x[1].transpose(1, 2)
    want = f64(q)
    q[:, 3, :, 77] = float("nan")
    masks = random_tree(n_q, 1, 9)
    out, lse = _tree(F, q, kd, vd, masks, T, cuda_dev)
    assert torch.isnan(out[:, 3].float()).all() and torch.isnan(lse[:, 3]).all()
    ok = [0, 1, 2, 4]
    khat, vhat = F.khat, F.vhat
    ref, lr = tree_reference(c, want, khat, vhat, f64(kd), f64(vd), masks, [T])
    vmax = np.abs(vhat).max()
    assert np.abs(f64(out)[:, ok] - ref[:, ok]).max() <= (2.0 ** -8 + 2.0 ** -10 + 2400 * 2.0 ** -28 + 1e-3) * vmax
    assert np.abs(f64(lse)[:, ok] - lr[:, ok]).max() <= 1e-3


@pytest.mark.parametrize("kb,G", [(2, 32), (4, 64), (8, 128), (16, 32)])
@pytest.mark.parametrize("si", range(len(SIZES) + 1))
def test_mass_scores_of_any_size(cuda_dev, kvq, si, kb, G):
    """Every weight within the error of its own score: the sum of a score's
    products in fp32 (2^-19 of their sizes) and the rounding of its exponent."""
    qs, ks = (SIZES + [([1e4], 1e-3)])[si]
    c = Case(1, 9, 3, 330, 13, 300, kb, 4, G, [1], konly=[2])
    n_q, T = 6, 321
    F, khat, _, q, _, _ = _scaled(c, 8400 + 10 * si, cuda_dev, n_q, qs, ks, 1.0)
    qf = f64(q)
    lse = np.zeros(qf.shape[:3], np.float32)
    for k in range(n_q):
        for hq in range(9):
            s = SCALE * (khat[0, hq // 3, :T - n_q + 1 + k] @ qf[0, k, hq])
            lse[0, k, hq] = s.max() + np.log(np.exp(s - s.max()).sum())
    mass = torch.full((1, 3, 330), -3.0, device=cuda_dev)
    kvq.attention_mass(F.L, F.cache, q, torch.from_numpy(lse).to(cuda_dev), T, mass, None, SCALE)
    torch.cuda.synchronize()
    want, tol = np.zeros((3, T)), np.zeros((3, T))
    se = score_error(qf, khat)
    for k in range(n_q):
        for hq in range(9):
            end = T - n_q + 1 + k
            w = np.exp(SCALE * (khat[0, hq // 3, :end] @ qf[0, k, hq]) - lse[0, k, hq])
            want[hq // 3, :end] += w
            tol[hq // 3, :end] += w * (2 * (se[0, k, hq] + 2.0 ** -21 * (1 + abs(lse[0, k, hq]))) + 2.0 ** -20)
    tol += 2.0 ** -22 * want + 1e-37
    err = np.abs(f64(mass)[0, :, :T] - want) / tol
    assert err.max() <= 1, f"mass: worst err / tol {err.max():.3g}"
    assert (mass[:, :, T:] == -3.0).all()


def test_mass_of_queries_past_fp16(cuda_dev, kvq):
    """Queries above 65504 (and keys so small that the scores are not)."""
    c = Case(1, 4, 2, 300, 10, 250, 4, 4, 64, [1])
    F, khat, _, q, _, _ = _scaled(c, 8600, cuda_dev, 1, [1.0], 1e-5, 1.0)
    q = (q.float() * 1e6).to(torch.bfloat16)
    qf = f64(q)
    s = np.stack([SCALE * (khat[0, hq // 2, :280] @ qf[0, 0, hq]) for hq in range(4)])
    lse = (s.max(1) + np.log(np.exp(s - s.max(1, keepdims=True)).sum(1))).astype(np.float32)
    mass = torch.zeros(1, 2, 300, device=cuda_dev)
    kvq.attention_mass(F.L, F.cache, q, torch.from_numpy(lse).to(cuda_dev).view(1, 1, 4), 280, mass, None, SCALE)
    torch.cuda.synchronize()
    w = np.exp(s - lse[:, None]).reshape(2, 2, 280).sum(1)
    rel = 2 * (score_error(qf, khat).max() + 2.0 ** -21 * (1 + np.abs(lse).max())) + 2.0 ** -19
    assert np.all(np.abs(f64(mass)[0, :, :280] - w) <= rel * w)


@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0, 1e-30])
def test_other_softmax_scales(cuda_dev, kvq, scale):
    """Zero (every position alike), negative, large and tiny scales."""
    c = Case(1, 6, 2, 330, 13, 300, 4, 4, 32, [1])
    F = Filled(c, 8700, cuda_dev)
    n_q, T = 5, 310
    q, x = bf16((1, n_q, 6, 128), 8701, cuda_dev), bf16((2, 1, n_q, 2, 128), 8702, cuda_dev)
    kd, vd = x[0].transpose(1, 2), x[1].transpose(1, 2)
    masks = np.array([[(1 << (i + 1)) - 1 for i in range(n_q)]], np.uint64)
    out, lse = torch.zeros_like(q), torch.zeros(1, n_q, 6, device=cuda_dev)
    ws = torch.zeros(kvq.decode_tree_workspace_bytes(F.L, n_q), dtype=torch.uint8, device=cuda_dev)
    kvq.decode_attention_tree(F.L, F.cache, q, kd, vd, masks_to(cuda_dev, masks), T, out, scale, lse, ws)
    kvq.quantize_append(F.L, F.cache, kd.contiguous(), vd.contiguous(), T)   # the chain behind its context
    mass = torch.zeros(1, 2, 330, device=cuda_dev)
    kvq.attention_mass(F.L, F.cache, q, lse, T + n_q, mass, None, scale)
    torch.cuda.synchronize()
    ref, lr = tree_reference(c, f64(q), F.khat, F.vhat, f64(kd), f64(vd), masks, [T], scale)
    se = score_error(f64(q), F.khat, f64(kd), abs(scale))
    vmax = max(np.abs(F.vhat).max(), np.abs(f64(vd)).max())
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 330 * 2.0 ** -28 + 2 * se[..., None]) * vmax
    assert (np.abs(f64(out) - ref) / tol).max() <= 1
    assert (np.abs(f64(lse) - lr) / (se + 2.0 ** -22 * (1 + np.abs(lr)))).max() <= 1
    # every token of the chain reaches what its lse is of: weights of 1 a query head
    total = f64(mass)[0, :, :T + n_q].sum(-1)
    assert np.abs(total - 3 * n_q).max() <= 3 * n_q * (4 * se.max() + 2.0 ** -18 * (1 + np.abs(lr).max()))
