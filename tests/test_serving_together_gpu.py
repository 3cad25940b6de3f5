"""The serving calls beside and after one another: evicted rows seen by a
decode that copies early, evictions in flight together against their own calls
alone, accepted root-to-node paths of the tree, waits that give up for
certain, and faint weights at the tree kernel's own resolution."""
import numpy as np
import pytest
import torch

import bit_mixed_precision_kvq_gb300 as kvq
from gpu_helpers import Case
from serving_ref import (SCALE, Filled, bf16, check_mass, f64, masks_to, random_tree, score_error, tree_reference)
from test_serving_flow_gpu import Loop, _grow

pytestmark = pytest.mark.gpu


def tight_tree(c, q, khat, vhat, kd, vd, masks, lens):
    """out, lse and their tolerances: as check_tree, with a faint weight off by
    2^-28 of the largest (P = 2^3 for the score that sets a reference, half a
    step of fp16's subnormals 2^-25)."""
    ref, lr = tree_reference(c, q, khat, vhat, kd, vd, masks, lens)
    g = c.H_q // c.H_kv
    se = score_error(q, khat, kd)
    vmax = np.repeat(np.maximum(np.abs(vhat).max(axis=(2, 3)), np.abs(vd).max(axis=(2, 3))), g, axis=1)[:, None, :, None]
    T = khat.shape[2] + q.shape[1]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + T * 2.0 ** -28 + 2 * se[..., None]) * vmax
    return ref, lr, tol, se + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(lr), lr, 0.0)))


def _tree_inputs(c, n_q, seed, dev):
    q, x = bf16((c.B, n_q, c.H_q, 128), seed, dev), bf16((2, c.B, n_q, c.H_kv, 128), seed + 1, dev)
    return q, x[0].transpose(1, 2), x[1].transpose(1, 2)


@pytest.mark.parametrize("c,n_q,T", [
    (Case(1, 8, 2, 9000, 14, 8900, 4, 2, 64, [0]), 6, 8950),
    (Case(2, 28, 4, 6400, 14, 14 + 6273, 4, 2, 64, [0]), 16, 6300),
], ids=str)
def test_tree_long_context_at_its_resolution(cuda_dev, kvq, c, n_q, T):
    F = Filled(c, 9000, cuda_dev)
    q, kd, vd = _tree_inputs(c, n_q, 9001, cuda_dev)
    masks = random_tree(n_q, 1, 4)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device=cuda_dev)
    ws = torch.zeros(kvq.decode_tree_workspace_bytes(F.L, n_q), dtype=torch.uint8, device=cuda_dev)
    kvq.decode_attention_tree(F.L, F.cache, q, kd, vd, masks_to(cuda_dev, masks), T, out, SCALE, lse, ws)
    torch.cuda.synchronize()
    ref, lr, tol, lt = tight_tree(c, f64(q), F.khat, F.vhat, f64(kd), f64(vd), masks, [T] * c.B)
    assert (np.abs(f64(out) - ref) / tol).max() <= 1
    assert (np.abs(f64(lse) - lr) / lt).max() <= 1


def test_tree_context_of_faint_weights(cuda_dev, kvq):
    """One position of every 128 outweighs the others by e^13.44 and holds
    zeros where they hold ones: the output is their share, within what 2^-28 of
    the largest weight allows a position (held next to a largest P of 1, their
    P would lie halfway between two steps of fp16 and be off by 2%)."""
    c = Case(1, 2, 1, 8200, 0, 0, 16, 16, 64, [])
    L = c.layout()
    T = 8000
    k = torch.zeros(1, 1, T, 128, dtype=torch.bfloat16, device=cuda_dev)
    v = torch.ones_like(k)
    k[:, :, ::128, 0], v[:, :, ::128] = 13.4375, 0.0
    cache = torch.zeros(int(L.total_bytes), dtype=torch.uint8, device=cuda_dev)
    kvq.quantize_append(L, cache, k, v, 0)
    q = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16, device=cuda_dev)
    q[..., 0] = 1.0 / SCALE
    kd = torch.full((1, 1, 1, 128), 3.0, dtype=torch.bfloat16, device=cuda_dev)   # attended by nobody
    gap = float(q[0, 0, 0, 0]) * SCALE * 13.4375
    out, lse = torch.zeros_like(q), torch.zeros(1, 1, 2, device=cuda_dev)
    ws = torch.zeros(kvq.decode_tree_workspace_bytes(L, 1), dtype=torch.uint8, device=cuda_dev)
    kvq.decode_attention_tree(L, cache, q, kd, kd, masks_to(cuda_dev, np.zeros((1, 1), np.uint64)), T, out, SCALE, lse, ws)
    torch.cuda.synchronize()
    loud = len(range(0, T, 128))
    w = (T - loud) * np.exp(-gap)
    want = w / (loud + w)
    assert np.all(np.abs(f64(out) - want) <= (2.0 ** -8 + 2.0 ** -10) * want + (T - loud) / loud * 2.0 ** -28)
    assert np.all(np.abs(f64(lse) - gap - np.log(loud + w)) <= 2.0 ** -19 * gap)


class PathLoop(Loop):
    """Loop whose accepted path is one drafted token's ancestors, root first."""

    def fill(self, seed, dev):
        m, path, n = super().fill(seed, dev)
        g = np.random.default_rng(seed + 1)
        path[:] = -1
        for b in range(self.F.c.B):
            node = int(g.integers(0, self.n_q))
            up = [j for j in range(self.n_q) if (int(m[b, node]) >> j) & 1][:self.max_path]
            n[b] = 0 if b == 1 else len(up)
            path[b, :n[b]] = up[:n[b]]
            for k, j in enumerate(path[b, :n[b]]):   # each accepted token sees those before it and itself
                assert int(m[b, j]) == sum(1 << int(i) for i in path[b, :k + 1])
        self.path.copy_(torch.from_numpy(path).to(dev))
        self.count.copy_(torch.from_numpy(n).to(dev))
        return m, path, n


def test_steps_along_root_to_node_paths(cuda_dev, kvq):
    """Tree, commit and mass with the path a verifier accepts: with the tree
    call's lse every accepted token's weights are a softmax, so a step adds
    g times the number of accepted tokens to the mass of a head."""
    c = Case(3, 8, 4, 500, 12, 400, 4, 2, 64, [0], konly=[2])
    F = Filled(c, 9100, cuda_dev)
    khat, vhat = F.khat.copy(), F.vhat.copy()
    lens, n_q, max_path, T = [420, 405, 460], 11, 8, 490
    loop = PathLoop(F, n_q, max_path, lens, cuda_dev)
    for s in range(3):
        m, path, n = loop.fill(9110 + 10 * s, cuda_dev)
        before = loop.mass.clone()
        loop.step(s % 2, T)
        torch.cuda.synchronize()
        kd, vd = f64(loop.kv[0].transpose(1, 2)), f64(loop.kv[1].transpose(1, 2))
        ref, lr, tol, lt = tight_tree(c, f64(loop.q), khat, vhat, kd, vd, m, lens)
        assert (np.abs(f64(loop.out) - ref) / tol).max() <= 1 and (np.abs(f64(loop.lse) - lr) / lt).max() <= 1
        _grow(F, khat, vhat, kd, vd, path, n, lens)
        lens = [lens[b] + int(n[b]) for b in range(3)]
        assert loop.len[1 - s % 2].tolist() == lens
        check_mass(c, loop.mass, f64(loop.q), f64(loop.lse), khat, lens, [list(path[b, :n[b]]) for b in range(3)],
                   f64(before), 0.95, before)
        added = (f64(loop.mass) - 0.95 * f64(before))
        for b in range(3):
            got = added[b, :, :lens[b]].sum(-1)
            assert np.abs(got - 2 * n[b]).max() <= 2e-3 * max(1, n[b])


def test_evicted_rows_are_seen_by_an_early_copying_decode(cuda_dev, kvq):
    """With kvq_set_cache_preload a decode copies cache rows before the
    previous kernel has finished: the rows that an eviction moved are there.
    Zero rows are appended in between, so that a row not yet moved shows."""
    c = Case(1, 28, 4, 1000, 14, 900, 4, 2, 64, [0])
    F = Filled(c, 9200, cuda_dev)
    D = Case(1, 28, 4, 700, 14, 614, 4, 2, 64, [0])
    Ld, T, T_dst = D.layout(), 960, 664
    dst = torch.zeros(int(Ld.total_bytes), dtype=torch.uint8, device=cuda_dev)
    mass = torch.rand(1, 4, 1000, device=cuda_dev)
    keep = torch.zeros(1, 4, T_dst, dtype=torch.int32, device=cuda_dev)
    zero = torch.zeros(1, 4, T_dst, 128, dtype=torch.bfloat16, device=cuda_dev)
    q = bf16((1, 28, 128), 9201, cuda_dev)
    ws = torch.zeros(int(Ld.workspace_bytes), dtype=torch.uint8, device=cuda_dev)
    out = [torch.zeros_like(q) for _ in range(3)]
    kvq.quantize_append(Ld, dst, zero, zero, 0)
    kvq.decode_attention(Ld, dst, q, T_dst, out[2], SCALE, None, ws)   # of zeros
    try:
        for r in range(20):
            for k, early in enumerate((False, True)):
                kvq.set_cache_preload(early)
                kvq.quantize_append(Ld, dst, zero, zero, 0)
                kvq.cache_evict(F.L, F.cache, mass, T, Ld, dst, T_dst, keep, 10)
                kvq.decode_attention(Ld, dst, q, T_dst, out[k], SCALE, None, ws)
            torch.cuda.synchronize()
            assert torch.equal(out[0], out[1])
            assert not out[2].any() and out[0].any()
    finally:
        kvq.set_cache_preload(False)


def test_calls_in_flight_together_equal_their_calls_alone(cuda_dev, kvq):
    """Tree, mass and eviction on two streams at once: outputs, masses, kept
    positions and moved rows are those of each alone."""
    c = Case(2, 8, 4, 3000, 10, 2900, 4, 2, 64, [0])
    F = Filled(c, 9300, cuda_dev)
    n_q, T = 16, 2950
    mask = masks_to(cuda_dev, random_tree(n_q, 1, 3))
    D = Case(2, 8, 4, 1100, 10, 1010, 4, 2, 64, [0]).layout()
    inputs = [_tree_inputs(c, n_q, 9310 + 5 * k, cuda_dev) for k in range(2)]

    def buffers():
        return (torch.zeros(2, n_q, 8, 128, dtype=torch.bfloat16, device=cuda_dev), torch.zeros(2, n_q, 8, device=cuda_dev),
                torch.zeros(2, 4, 3000, device=cuda_dev), torch.zeros(int(D.total_bytes), dtype=torch.uint8, device=cuda_dev),
                torch.zeros(2, 4, 1040, dtype=torch.int32, device=cuda_dev),
                torch.zeros(kvq.decode_tree_workspace_bytes(F.L, n_q), dtype=torch.uint8, device=cuda_dev))

    def work(k, to, stream=None):
        q, kd, vd = inputs[k]
        out, lse, mass, dst, keep, ws = to
        kvq.decode_attention_tree(F.L, F.cache, q, kd, vd, mask, T, out, SCALE, lse, ws, stream=stream)
        kvq.attention_mass(F.L, F.cache, q, lse, T, mass, None, SCALE, stream=stream)
        kvq.cache_evict(F.L, F.cache, mass, T, D, dst, 1040, keep, 10, stream=stream)

    alone = [buffers() for _ in range(2)]
    for k in range(2):
        work(k, alone[k])
        torch.cuda.synchronize()
    rounds = [[buffers() for _ in range(2)] for _ in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for r in range(4):
        for k in range(2):
            work(k, rounds[r][k], streams[k])
    torch.cuda.synchronize()
    for r in range(4):
        for k in range(2):
            for got, want in zip(rounds[r][k][:5], alone[k][:5]):
                assert torch.equal(got, want)


@pytest.mark.parametrize("c,T", [
    (Case(2, 8, 2, 2000, 10, 1900, 4, 2, 64, [0]), 1950),     # split units: marks pass through the partials
    (Case(2, 8, 2, 200, 10, 150, 4, 2, 64, [0]), 100),        # one CTA per unit
], ids=str)
def test_waits_give_up_for_certain(cuda_dev, kvq, c, T):
    """A limit of one poll asks once, without suspending: the first wait on
    the queries gives up.  The status is set, every row is either right or NaN
    as a whole, some are NaN, and the next call is right again."""
    F = Filled(c, 9400, cuda_dev)
    n_q = 12
    q, kd, vd = _tree_inputs(c, n_q, 9401, cuda_dev)
    m = random_tree(n_q, 1, 5)
    mask = masks_to(cuda_dev, m)
    out, lse = torch.zeros_like(q), torch.zeros(2, n_q, 8, device=cuda_dev)
    ws = torch.zeros(kvq.decode_tree_workspace_bytes(F.L, n_q), dtype=torch.uint8, device=cuda_dev)
    ref, lr, tol, lt = tight_tree(c, f64(q), F.khat, F.vhat, f64(kd), f64(vd), m, [T, T])

    def rows():
        o, l = f64(out), f64(lse)
        nan = np.isnan(l)
        assert np.array_equal(np.isnan(o), np.repeat(nan[..., None], 128, -1))
        assert np.all(np.abs(o - ref)[~nan] <= tol[~nan]) and np.all(np.abs(l - lr)[~nan] <= lt[~nan])
        return int(nan.sum())

    try:
        kvq.set_wait_limits(1, 0)
        kvq.decode_attention_tree(F.L, F.cache, q, kd, vd, mask, T, out, SCALE, lse, ws)
        torch.cuda.synchronize()
    finally:
        kvq.set_wait_limits(0, 0)
    assert kvq.workspace_status(ws) == kvq.STATUS_TILE_WAIT
    assert rows() > 0
    ws.zero_()
    kvq.decode_attention_tree(F.L, F.cache, q, kd, vd, mask, T, out, SCALE, lse, ws)
    torch.cuda.synchronize()
    assert kvq.workspace_status(ws) == 0 and rows() == 0
