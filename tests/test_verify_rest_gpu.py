"""kvq_tree_verify where refused siblings hold nearly all of the probability:
what they leave is held against random numbers next to their borders.  Tiny temperatures."""
import numpy as np
import pytest
import torch

from step_ref import check_verify, verify_reference
from test_tree_verify_gpu import run

pytestmark = pytest.mark.gpu


class Rest:
    """Token 0 with n - 1 children; child k's probability is 1 - left[k] of what
    its earlier siblings leave.  All but the last are refused whatever their probability (NaN
    numbers, or `u`); the last one's number lies next to its border."""

    def __init__(self, B, n, V, half, left, side, seed, u=np.nan):
        g = np.random.default_rng(seed)
        x = g.normal(0, 1, (B, n, V)).astype(np.float32)
        ids = np.stack([g.permutation(V)[:n] for _ in range(B)])
        self.masks = np.array([[1] + [1 | (1 << j) for j in range(1, n)]], np.uint64)
        self.tokens = np.zeros((B, n), np.int32)
        self.tokens[:, 1:] = ids[:, 1:]
        for b in range(B):
            rest = np.delete(x[b, 0].astype(np.float64), ids[b, 1:])
            mass = np.exp(rest).sum() * 4.0  # of the rest and the last child
            x[b, 0, ids[b, n - 1]] = np.log(mass * 0.75)
            for k in range(n - 2, 0, -1):
                x[b, 0, ids[b, k]] = np.log(mass * (1 / left[k - 1] - 1))
                mass /= left[k - 1]
        self.t = torch.from_numpy(x)
        if half:
            self.t = self.t.bfloat16()
        self.x = self.t.float().numpy()
        self.draft = None
        self.race = g.exponential(size=(B, V)).astype(np.float32)
        self.u = np.full((B, n), u, np.float32)
        for b in range(B):
            p = np.exp(self.x[b, 0].astype(np.float64) - self.x[b, 0].max())
            p[ids[b, 1:n - 1]] = 0
            border = p[ids[b, n - 1]] / p.sum()
            # 2^-10 of the border to either side: fp32 decides what is 2^-14 from it
            self.u[b, n - 1] = np.float32(border * (1 + side[b % len(side)] * 2.0 ** -10))


@pytest.mark.parametrize("V", [40, 5003, 150001])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("left", [[1e-3], [1e-5], [3e-6], [4e-7], [0.5], [1e-3, 1e-3], [2e-6, 0.3], [0.5, 1e-5], [1e-5, 1e-5], [0.3, 0.3, 1e-4, 1e-4], [1e-6, 1e-6, 0.5]])
def test_borders_behind_refused_siblings(cuda_dev, kvq, left, half, V):
    s = Rest(6, len(left) + 2, V, half, left, [-1, 1], 300 + V)
    ref = verify_reference(s.x, s.tokens, s.masks, s.u, s.race)
    last = len(left) + 1
    assert all(ref[0][b][1] == (last if b % 2 == 0 else -1) for b in range(6))  # (the reference decides as meant)
    check_verify(run(kvq, cuda_dev, s), ref, scores=128.0)


@pytest.mark.parametrize("V", [40, 5003, 150001])
@pytest.mark.parametrize("left", [1e-3, 1e-5, 3e-6, 4e-7])
def test_the_largest_number_refuses_a_near_certain_child(cuda_dev, kvq, left, V):
    """u = 1 - 2^-24 refuses p = 1 - left.  In fp32 p = 1 / (1 + s) is off by
    2^-23 and a rounding of u * 1 by none: 1.2e-7 of the 3.4e-7 and more between them, so the
    decision is certain, although nearer to its border than 2^-14."""
    s = Rest(4, 3, V, False, [left], [-1, 1], 320 + V, 1 - 2.0 ** -24)
    path, plen, nxt, logp, _ = verify_reference(s.x, s.tokens, s.masks, s.u, s.race)
    out = run(kvq, cuda_dev, s)
    assert plen.tolist() == [2, 1, 2, 1] and np.array_equal(out[0].cpu().numpy(), path) and np.array_equal(out[1].cpu().numpy(), plen)
    for b in range(4):  # the pick, where the two largest keys are 2^-14 apart
        row = 2 if b % 2 == 0 else 0
        x = s.x[b, row].astype(np.float64)
        p = np.exp(x - x.max())
        if row == 0:
            p[s.tokens[b, 1:]] = 0
        two = np.sort(p / s.race[b])[-2:]
        assert two[0] >= two[1] * (1 - 2.0 ** -14) or int(out[2][b]) == nxt[b]


@pytest.mark.parametrize("V", [9, 20011])
def test_refused_siblings_in_any_order(cuda_dev, kvq, V):
    """The largest token refused last; ties of the largest; a NaN number refuses all of the mass."""
    s = Rest(4, 5, V, False, [1e-4, 1e-4, 0.4], [-1, 1], 310)
    order = [2, 3, 1]
    for b in (0, 1):
        s.tokens[b, 1:4] = s.tokens[b, order]
        s.u[b, 1:4] = np.nan  # refused whatever their probability
    for b in (2, 3):  # two equal largest ones, the higher id refused first
        pair = sorted(s.tokens[b, 1:3], reverse=True)
        s.tokens[b, 1:3] = pair
        s.x[b, 0, pair] = s.x[b, 0].max()
        s.u[b, 1:3] = np.nan
        p = np.exp(s.x[b, 0].astype(np.float64) - s.x[b, 0].max())
        p[s.tokens[b, 1:4]] = 0
        s.u[b, 4] = np.float32(p[s.tokens[b, 4]] / p.sum() * (1 + (-1) ** b * 2.0 ** -10))
        s.u[b, 3] = np.nan
    s.t = torch.from_numpy(s.x)
    check_verify(run(kvq, cuda_dev, s), verify_reference(s.x, s.tokens, s.masks, s.u, s.race), scores=128.0)


def test_nothing_left(cuda_dev, kvq):
    """One token holds all of the probability and is refused: no sibling is taken, and it is picked."""
    s = Rest(3, 4, 777, False, [0.5, 0.5], [1], 311)
    for b in range(3):
        s.x[b, 0] = -np.inf
        s.x[b, 0, s.tokens[b, 1]] = 3.0
    s.u[:, 1] = np.nan
    s.u[:, 2:] = 0.0
    s.t = torch.from_numpy(s.x)
    out = run(kvq, cuda_dev, s)
    assert out[1].tolist() == [1, 1, 1] and out[2].tolist() == s.tokens[:, 1].tolist()


def test_tiny_temperatures(cuda_dev, kvq):
    """Temperatures whose inverse leaves fp32, with logits that stay finite over them."""
    s = Rest(4, 3, 3001, False, [0.5], [1], 312)
    s.x[:] = np.random.default_rng(313).integers(-3, 1, s.x.shape) * np.float32(2.0 ** -4)
    s.t = torch.from_numpy(s.x)
    heat = [2e-39, 1e-39, 1e-38, 4e-39]
    check_verify(run(kvq, cuda_dev, s, heat), verify_reference(s.x, s.tokens, s.masks, s.u, s.race, None, heat))
