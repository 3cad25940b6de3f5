"""64-bit references of the tree, commit, mass and eviction calls (numpy over
the oracle's reconstruction of the cache), their tolerances, and helpers that
make the inputs of a case."""
from __future__ import annotations

import numpy as np
import torch

import oracle
import synth
from gpu_helpers import Case, alloc_cache, append, bits

SCALE = 1.0 / np.sqrt(128.0)


def bf16(shape, seed, dev, scale=1.0):
    n = int(np.prod(shape))
    return synth.to_bf16(scale * synth.normal(n, synth.stream_key(seed, 21), dev)).view(*shape)


def f64(x: torch.Tensor) -> np.ndarray:
    return x.detach().to("cpu").to(torch.float64).numpy()


class Filled:
    """A case's cache, filled from seeded rows, and the values it stands for."""

    def __init__(self, c: Case, seed: int, dev, fill: int = 0xA5):
        self.c, self.L = c, c.layout()
        self.k, self.v = bf16((c.B, c.H_kv, c.T_cap, c.D), seed, dev), bf16((c.B, c.H_kv, c.T_cap, c.D), seed + 1, dev)
        self.cache = alloc_cache(self.L, dev, fill)
        append(self.L, self.cache, self.k, self.v, 0)
        self.khat = oracle.reconstruct(bits(self.k), c.vs, c.ve, c.mask(), c.kb, c.G)[0]
        m = [1 if x == 1 else 0 for x in c.mask()]  # a K-only head's V is quantised
        self.vhat = oracle.reconstruct(bits(self.v), c.vs, c.ve, m, c.vb, c.G)[0]


def random_tree(n_q: int, rows: int, seed: int, reach: int = 6) -> np.ndarray:
    """Ancestor masks (own bit included) of random trees, uint64 [rows, n_q]."""
    g = np.random.default_rng(seed)
    m = np.zeros((rows, n_q), np.uint64)
    for b in range(rows):
        for i in range(n_q):
            p = int(g.integers(max(-1, i - reach), i)) if i else -1
            m[b, i] = (m[b, p] if p >= 0 else np.uint64(0)) | np.uint64(1 << i)
    return m


def masks_to(dev, m: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(m).view(np.int64)).to(dev)


def tree_reference(c: Case, q, khat, vhat, kd, vd, masks, lens, scale=SCALE):
    """out [B, n_q, H_q, D], lse [B, n_q, H_q] (lens[b] None: inactive)."""
    B, n_q, Hq, D = q.shape
    g = c.H_q // c.H_kv
    out, lse = np.zeros(q.shape), np.full((B, n_q, Hq), -np.inf)
    for b in range(B):
        if lens[b] is None:
            continue
        n = lens[b]
        sees = np.ones((n_q, n + n_q), bool)
        for i in range(n_q):
            for j in range(n_q):
                sees[i, n + j] = (int(masks[b % len(masks), i]) >> j) & 1
        for h in range(c.H_kv):
            k = np.concatenate([khat[b, h, :n], kd[b, h]])
            v = np.concatenate([vhat[b, h, :n], vd[b, h]])
            for i in range(n_q):
                at = np.nonzero(sees[i])[0]
                if not len(at):
                    continue
                s = scale * (k[at] @ q[b, i, h * g:(h + 1) * g].T)       # [rows, g]
                top = s.max(0)
                e = np.exp(s - top)
                lse[b, i, h * g:(h + 1) * g] = top + np.log(e.sum(0))
                out[b, i, h * g:(h + 1) * g] = (e / e.sum(0)).T @ v[at]
    return out, lse


def score_error(q, khat, kd=None, scale=SCALE):
    """Bound of a score's error, [B, n_q, H_q]: the operands are exact, the
    products accumulate in fp32 over at most 16 steps of a tensor-core or
    shuffle sum, each off by at most 2^-23 of the running magnitude (a
    truncating adder), i.e. 2^-19 in all; a running magnitude is at most
    sum |q_d| (|code * s| + |z|) <= 3 max|K| sum |q_d|."""
    B, n_q, Hq, _ = q.shape
    H = khat.shape[1]
    kmax = np.abs(khat).max(axis=(2, 3))                                # [B, H]
    if kd is not None:
        kmax = np.maximum(kmax, np.abs(kd).max(axis=(2, 3)))
    return 2.0 ** -19 * scale * np.abs(q).sum(-1) * 3 * np.repeat(kmax, Hq // H, axis=1)[:, None, :]


def check_tree(c: Case, out, lse, q, khat, vhat, kd, vd, masks, lens, scale=SCALE):
    """out: one bf16 rounding, 2^-8 of the value; P and (dequantised) V held
    in fp16, 2^-11 each; a P below the normal range of fp16 is off by at most
    2^-25 of the largest one, per position; a score's error e moves a weight
    by a factor of e^(2e).  lse: the score error and fp32 roundings."""
    ref, lr = tree_reference(c, q, khat, vhat, kd, vd, masks, lens, scale)
    T = khat.shape[2] + q.shape[1]
    g = c.H_q // c.H_kv
    se = score_error(q, khat, kd, scale)
    vmax = np.maximum(np.abs(vhat).max(axis=(2, 3)), np.abs(vd).max(axis=(2, 3)))
    vmax = np.repeat(vmax, g, axis=1)[:, None, :, None]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + T * 2.0 ** -25 + 2 * se[..., None]) * vmax
    o = f64(out)
    assert np.all(np.isfinite(o))
    err = np.abs(o - ref)
    assert np.all(err <= tol), f"out: worst err / tol {np.max(err / tol):.3g}"
    worst = float(np.max(err / tol))
    if lse is not None:
        l = f64(lse)
        assert np.array_equal(np.isneginf(l), np.isneginf(lr))
        fin = np.isfinite(lr)
        le, lt = np.abs(l[fin] - lr[fin]), se[fin] + 2.0 ** -22 * (1 + np.abs(lr[fin]))
        assert np.all(le <= lt), f"lse: worst err / tol {np.max(le / lt):.3g}"
    return worst


def mass_reference(c: Case, q, lse, khat, lens, taken, mass_in, decay, scale=SCALE):
    """mass for t < lens[b] (NaN elsewhere and for inactive sequences), and
    the summed weights."""
    B = q.shape[0]
    g = c.H_q // c.H_kv
    mass = np.full((B, c.H_kv, c.T_cap), np.nan)
    add = np.zeros((B, c.H_kv, c.T_cap))
    for b in range(B):
        if lens[b] is None:
            continue
        n, toks = lens[b], taken[b]
        for h in range(c.H_kv):
            w = np.zeros(n)
            for k, tok in enumerate(toks):
                end = n - len(toks) + 1 + k
                for hq in range(h * g, (h + 1) * g):
                    l = lse[b, tok, hq]
                    if np.isfinite(l):
                        w[:end] += np.exp(scale * (khat[b, h, :end] @ q[b, tok, hq]) - l)
            add[b, h, :n] = w
            mass[b, h, :n] = w + (decay * mass_in[b, h, :n] if mass_in is not None else 0.0)
    return mass, add


def check_mass(c: Case, got, q, lse, khat, lens, taken, mass_in, decay, before, scale=SCALE):
    """Every term e^(s - lse) is off by the score error and the fp32 rounding
    of its exponent (2^-23 of |s| + |lse|, times 2 for the two operations in
    log2 units); sums of at most 2^9 terms in fp32.  Positions that are not
    written keep their bits."""
    ref, add = mass_reference(c, q, lse, khat, lens, taken, mass_in, decay, scale)
    o = f64(got)
    written = ~np.isnan(ref)
    assert np.array_equal(got.cpu().numpy()[~written], before.cpu().numpy()[~written])
    se = score_error(q, khat, scale=scale).max()
    fin = np.abs(lse[np.isfinite(lse)])
    rel = 2 * (se + 2.0 ** -21 * (1 + (fin.max() if fin.size else 0.0))) + 2.0 ** -20
    tol = rel * add + 2.0 ** -22 * np.abs(np.nan_to_num(ref)) + 1e-37
    err = np.abs(o - ref)[written]
    assert np.all(err <= tol[written]), f"mass: worst err / tol {np.max(err / tol[written]):.3g}"


def keep_reference(c: Case, mass: np.ndarray, lens, k_vis: int, k_text: int, recent: int) -> np.ndarray:
    """Kept source positions [B, H_kv, vs + k_vis + k_text], -1 behind the last."""
    x = np.where(np.isnan(mass), -np.inf, mass.astype(np.float64))
    # NaN below every number, -inf included: a second key
    low = np.isnan(mass)
    keep = np.full((mass.shape[0], c.H_kv, c.vs + k_vis + k_text), -1, np.int64)

    def best(b, h, at, n):
        order = np.lexsort((at, -np.nan_to_num(x[b, h, at], neginf=-1e300, posinf=1e300), low[b, h, at]))
        return np.sort(at[order[:n]])

    for b in range(mass.shape[0]):
        if lens[b] is None:
            continue
        n = lens[b]
        for h in range(c.H_kv):
            old = max(c.ve, n - recent)
            at = np.concatenate([np.arange(c.vs), best(b, h, np.arange(c.vs, c.ve), k_vis),
                                 best(b, h, np.arange(c.ve, old), max(0, k_text - (n - old))), np.arange(old, n)])
            keep[b, h, :len(at)] = at
    return keep
