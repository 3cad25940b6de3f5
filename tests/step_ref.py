"""64-bit references and tolerances of the norm-and-rotation, tree-verification
and windowed decode calls."""
from __future__ import annotations

import numpy as np
import torch

from serving_ref import SCALE, f64, score_error


def rope_reference(x, pos, freq, axis, rot, interleaved, weight, eps):
    """x [B, n, H, D], pos [n_axes, B, n]: y of kvq_norm_rope in 64 bits, and the
    size |y_p| + |y_q| of each element's pair (|y| beyond the rotated part)."""
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * weight
    i = np.arange(rot // 2)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    angle = np.moveaxis(pos[np.asarray(axis)].astype(np.float64), 0, -1) * freq   # [B, n, rot / 2]
    c, s = np.cos(angle)[:, :, None], np.sin(angle)[:, :, None]
    out, size = y.copy(), np.abs(y)
    out[..., p] = y[..., p] * c - y[..., q] * s
    out[..., q] = y[..., q] * c + y[..., p] * s
    size[..., p] = size[..., q] = np.abs(y[..., p]) + np.abs(y[..., q])
    return out, size


def check_rope(got, x, pos, freq, axis, rot, interleaved, weight, eps):
    """One bf16 rounding (2^-8 of the value as computed).  Before it, relative
    to the pair: the norm's sum of 128 squares over 8 sequential and 4 shuffled
    additions, its root (2 units) and two products: 2^-20; the angle to 2^-25
    of a turn (6.3 * 2^-25 < 2^-22), sincospi to 2^-22, two products and a sum:
    2^-21.  2^-19 in all, and bf16 subnormals are steps of 2^-133."""
    ref, size = rope_reference(x, pos, freq, axis, rot, interleaved, weight, eps)
    tol = (2.0 ** -8 * (1 + 2.0 ** -8)) * np.abs(ref) + 2.0 ** -18 * size + 2.0 ** -133
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), f"worst err / tol {np.max(err / tol):.3g}"


def parents_of(masks: np.ndarray) -> np.ndarray:
    """Highest set bit below the token's own, -1 without one; masks uint64 [rows, n]."""
    par = np.full(masks.shape, -1, np.int64)
    for r in range(masks.shape[0]):
        for j in range(masks.shape[1]):
            below = int(masks[r, j]) & ((1 << j) - 1)
            par[r, j] = below.bit_length() - 1
    return par


def verify_reference(logits, tokens, masks, u, race, draft=None, heat=None, size=None):
    """Walk of every tree in 64 bits: (path, path_len, next, logprob, margin);
    margin: how far, relative to its larger side, the nearest decision was from
    its border (a score within 2^-14 of it may fall either way in 32 bits)."""
    B, n, V = logits.shape
    path, plen = np.full((B, n), -1, np.int64), np.full(B, -1, np.int64)
    nxt, logp, margin = np.full(B, -1, np.int64), np.zeros((B, n)), np.full(B, np.inf)
    par = parents_of(masks)
    for b in range(B):
        m = n if size is None else int(size[b])
        if not 1 <= m <= n:
            continue
        t = 1.0 if heat is None else float(heat[b])
        greedy = not t > 0
        walk, lps, cur, bad = [0], [], 0, False
        while True:
            x = logits[b, cur].astype(np.float64) / (1.0 if greedy else t)
            if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
                bad = True
                break
            lp = x - x.max()
            lp = lp - np.log(np.exp(lp).sum())
            best = int(np.argmax(x))
            p, gone, goes = np.exp(lp), set(), None
            q = None if draft is None else draft[b, cur].astype(np.float64)
            for j in range(1, m):
                if par[b % len(masks), j] != cur:
                    continue
                c = int(tokens[b, j])
                known = 0 <= c < V
                if greedy:
                    ok = c == best
                elif not known:
                    ok = False
                else:
                    total = p.sum()
                    have, want = p[c], float(u[b, j]) * total * (1.0 if q is None else q[c])
                    ok = have > 0 and want < have
                    if c not in gone or q is not None:
                        margin[b] = min(margin[b], abs(have - want) / max(have, want, 1e-300))
                if ok:
                    goes = j
                    break
                if greedy:
                    continue
                if q is not None:
                    r = np.fmax(p / p.sum() - q, 0)
                    if r.sum() > 0:
                        p = r
                elif known:
                    p[c] = 0.0
                    gone.add(c)
            if goes is None:
                break
            lps.append(lp[int(tokens[b, goes])])
            walk.append(goes)
            cur = goes
        if bad:
            margin[b] = np.inf
            continue
        nxt[b] = best
        if not greedy:
            e = race[b].astype(np.float64)
            key = np.where(e > 0, p / np.where(e > 0, e, 1), 0)
            if key.max() > 0:
                nxt[b] = int(np.argmax(key))
                top = np.sort(key)[-2:]
                if V > 1:
                    margin[b] = min(margin[b], (top[1] - top[0]) / top[1])
        lps.append(lp[nxt[b]])
        path[b, :len(walk)], plen[b], logp[b, :len(walk)] = walk, len(walk), lps
    return path, plen, nxt, logp, margin


def check_verify(out, ref, scores: float = 64.0):
    """Whole values equal wherever every decision lies 2^-14 from its border.
    logprob: the exponent's argument in fp32, 3 roundings of at most `scores`
    (2^-22 of it), and a sum of exponentials off by 2^-17 (at most 2^5
    sequential additions and 2^5 joins, 2^-22 for an exponential of a weight
    that counts)."""
    path, plen, nxt, logp, margin = ref
    sure = margin > 2.0 ** -14
    assert sure.mean() > 0.8, "too many borderline sequences to say anything"
    got = [x.cpu().numpy() for x in out]
    for a, b in zip(got[:3], (path, plen, nxt)):
        assert np.array_equal(a[sure], b[sure])
    if got[3] is not None:
        err = np.abs(got[3][sure].astype(np.float64) - logp[sure])
        tol = np.where(path[sure] >= 0, 2.0 ** -17 + 2.0 ** -22 * scores + 2.0 ** -23 * np.abs(logp[sure]), 0.0)
        assert np.all(err <= tol), f"logprob: worst err / tol {np.max(err / np.maximum(tol, 1e-300)):.3g}"


def window_reference(c, q, khat, vhat, lens, n_sink, window, scale=SCALE):
    """out [B, n_q, H_q, D], lse [B, n_q, H_q] (lens[b] None: inactive)."""
    B, n_q, Hq, D = q.shape
    g = c.H_q // c.H_kv
    out, lse = np.zeros(q.shape), np.full((B, n_q, Hq), -np.inf)
    for b in range(B):
        if lens[b] is None:
            continue
        for i in range(n_q):
            p = lens[b] - n_q + i
            t = np.arange(max(0, p + 1))
            t = t[(t < n_sink) | (t > p - window)]
            if not len(t):
                continue
            for h in range(c.H_kv):
                s = scale * (khat[b, h, t] @ q[b, i, h * g:(h + 1) * g].T)
                top = s.max(0)
                e = np.exp(s - top)
                lse[b, i, h * g:(h + 1) * g] = top + np.log(e.sum(0))
                out[b, i, h * g:(h + 1) * g] = (e / e.sum(0)).T @ vhat[b, h, t]
    return out, lse


def check_window(c, out, lse, q, khat, vhat, lens, n_sink, window, scale=SCALE, codes=True):
    """out: one bf16 rounding, 2^-8 of the value; a packed row's weight is
    rounded to fp16 and again as it meets its scale, 2^-11 each, the second of
    code * scale <= 2 max|V| (3 * 2^-11 max|V| in all); weights of bf16 rows
    to 2^-17.  What a weight loses below fp16's normal range is 2^-25 of steps
    whose largest weight is 2^11 or more (2^-8 where a scale reaches 2^12):
    scale * weight off by 2^-25 times a code of at most 255, 2^-17 * 2^-11 for a
    position (codes False: all of them are 0), and the weight itself 2^-36.  A score's error e moves a weight by a
    factor of e^(2e).  lse: the score error and fp32 roundings."""
    ref, lr = window_reference(c, q, khat, vhat, lens, n_sink, window, scale)
    rows = min(khat.shape[2], n_sink + window + q.shape[1])
    g = c.H_q // c.H_kv
    se = score_error(q, khat, scale=abs(scale))
    vmax = np.repeat(np.abs(vhat).max(axis=(2, 3)), g, axis=1)[:, None, :, None]
    tol = 2.0 ** -8 * np.abs(ref) + (3 * 2.0 ** -11 + 2 * se[..., None]) * vmax + (rows * 2.0 ** -28 * np.maximum(1, vmax) if codes else 0)
    o = f64(out)
    assert np.all(np.isfinite(o))
    err = np.abs(o - ref)
    assert np.all(err <= tol), f"out: worst err / tol {np.max(err / tol):.3g}"
    if lse is not None:
        l = f64(lse)
        assert np.array_equal(np.isneginf(l), np.isneginf(lr))
        fin = np.isfinite(lr)
        le, lt = np.abs(l[fin] - lr[fin]), se[fin] + 2.0 ** -21 * (1 + np.abs(lr[fin]))
        assert np.all(le <= lt), f"lse: worst err / tol {np.max(le / lt):.3g}"
    return float(np.max(err / tol))
