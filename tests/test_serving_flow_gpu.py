"""The tree, commit, mass and eviction calls as a decode loop runs them:
several steps on device lengths, captured and replayed, on other streams,
with another call's work in flight, and with waits that give up."""
import numpy as np
import pytest
import torch

import bit_mixed_precision_kvq_gb300 as kvq
from gpu_helpers import Case, bits
from serving_ref import (SCALE, Filled, bf16, check_mass, check_tree, f64, keep_reference, masks_to, random_tree,
                         tree_reference)

pytestmark = pytest.mark.gpu


class Loop:
    """Buffers of a loop that drafts n_q tokens a step."""

    def __init__(self, F, n_q, max_path, lens, dev):
        c = F.c
        self.F, self.n_q, self.max_path = F, n_q, max_path
        self.q = torch.zeros(c.B, n_q, c.H_q, 128, dtype=torch.bfloat16, device=dev)
        self.kv = torch.zeros(2, c.B, n_q, c.H_kv, 128, dtype=torch.bfloat16, device=dev)
        self.mask = torch.zeros(c.B, n_q, dtype=torch.int64, device=dev)
        self.path = torch.zeros(c.B, max_path, dtype=torch.int32, device=dev)
        self.count = torch.zeros(c.B, dtype=torch.int32, device=dev)
        self.len = [torch.tensor(lens, dtype=torch.int32, device=dev), torch.zeros(c.B, dtype=torch.int32, device=dev)]
        self.out = torch.zeros_like(self.q)
        self.lse = torch.zeros(c.B, n_q, c.H_q, device=dev)
        self.mass = torch.zeros(c.B, c.H_kv, c.T_cap, device=dev)
        self.ws = torch.zeros(kvq.decode_tree_workspace_bytes(F.L, n_q), dtype=torch.uint8, device=dev)

    def fill(self, seed, dev):
        """A step's inputs: drafts, their tree, and an accepted path of it."""
        c, n_q = self.F.c, self.n_q
        self.q.copy_(bf16(self.q.shape, seed, dev))
        self.kv.copy_(bf16(self.kv.shape, seed + 1, dev))
        m = random_tree(n_q, c.B, seed, reach=4)
        self.mask.copy_(masks_to(dev, m))
        g = np.random.default_rng(seed)
        path = np.full((c.B, self.max_path), -1, np.int32)
        n = np.zeros(c.B, np.int32)
        for b in range(c.B):  # the ancestors of a drafted token, from the root down
            up = [j for j in range(n_q) if (int(m[b, int(g.integers(0, n_q))]) >> j) & 1][:self.max_path]
            n[b] = 0 if g.random() < 0.2 else len(up)
            path[b, :n[b]] = up[:n[b]]
        self.path.copy_(torch.from_numpy(path).to(dev))
        self.count.copy_(torch.from_numpy(n).to(dev))
        return m, path, n

    def step(self, k, T):
        """One step from the lengths len[k] to len[1 - k]."""
        F, old, new = self.F, self.len[k], self.len[1 - k]
        kd, vd = self.kv[0].transpose(1, 2), self.kv[1].transpose(1, 2)
        kvq.decode_attention_tree(F.L, F.cache, self.q, kd, vd, self.mask, T, self.out, SCALE, self.lse, self.ws, seq_len=old)
        kvq.tree_commit(F.L, F.cache, kd, vd, self.path, self.count, T, seq_len=old, new_len=new)
        kvq.attention_mass(F.L, F.cache, self.q, self.lse, T + self.max_path, self.mass, self.mass, SCALE, 0.95, seq_len=new,
                           path=self.path, path_len=self.count)


def _grow(F, khat, vhat, kd, vd, path, n, lens):
    """The committed rows in the reference's values."""
    for b in range(F.c.B):
        for k in range(n[b]):
            khat[b, :, lens[b] + k], vhat[b, :, lens[b] + k] = kd[b, :, path[b, k]], vd[b, :, path[b, k]]


def test_speculative_steps_then_eviction(cuda_dev, kvq):
    """Three steps of tree, commit and mass on device lengths, then an
    eviction, then a tree step and a plain decode on the smaller cache."""
    c = Case(3, 8, 4, 500, 12, 400, 4, 2, 64, [0], konly=[2])
    F = Filled(c, 7000, cuda_dev)
    khat, vhat = F.khat.copy(), F.vhat.copy()
    lens, n_q, max_path, T = [420, 405, 460], 11, 5, 480
    loop = Loop(F, n_q, max_path, lens, cuda_dev)
    mass = np.zeros((3, 4, 500))
    for s in range(3):
        m, path, n = loop.fill(7100 + 10 * s, cuda_dev)
        before = loop.mass.clone()
        loop.step(s % 2, T)
        torch.cuda.synchronize()
        assert kvq.workspace_status(loop.ws) == 0
        kd, vd = f64(loop.kv[0].transpose(1, 2)), f64(loop.kv[1].transpose(1, 2))
        check_tree(c, loop.out, loop.lse, f64(loop.q), khat, vhat, kd, vd, m, lens)
        _grow(F, khat, vhat, kd, vd, path, n, lens)
        lens = [lens[b] + int(n[b]) for b in range(3)]
        assert loop.len[1 - s % 2].tolist() == lens
        taken = [list(path[b, :n[b]]) for b in range(3)]
        check_mass(c, loop.mass, f64(loop.q), f64(loop.lse), khat, lens, taken, f64(before), 0.95, before)
    # eviction: 150 visual and 40 text positions per head stay
    D = Case(3, 8, 4, 260, 12, 162, 4, 2, 64, [0], konly=[2])
    Ld, T_dst = D.layout(), 202
    dst = torch.zeros(int(Ld.total_bytes), dtype=torch.uint8, device=cuda_dev)
    keep = torch.zeros(3, 4, T_dst, dtype=torch.int32, device=cuda_dev)
    mass_dst = torch.zeros(3, 4, 260, device=cuda_dev)
    new = torch.zeros(3, dtype=torch.int32, device=cuda_dev)
    now = loop.len[1]
    kvq.cache_evict(F.L, F.cache, loop.mass, T + max_path, Ld, dst, T_dst, keep, 8, mass_dst, now, new)
    torch.cuda.synchronize()
    at = keep_reference(c, loop.mass.cpu().numpy(), lens, 150, 40, 8)
    assert np.array_equal(keep.cpu().numpy(), at)
    ends = [12 + 150 + min(40, n - 400) for n in lens]
    assert new.tolist() == ends
    k2, v2 = np.zeros((3, 4, 260, 128)), np.zeros((3, 4, 260, 128))
    for b in range(3):
        for h in range(4):
            k2[b, h, :ends[b]], v2[b, h, :ends[b]] = khat[b, h, at[b, h, :ends[b]]], vhat[b, h, at[b, h, :ends[b]]]
    G = type("Smaller", (), dict(c=D, L=Ld, cache=dst))
    loop2 = Loop(G, n_q, max_path, ends, cuda_dev)
    loop2.mass.copy_(mass_dst)
    m, path, n = loop2.fill(7200, cuda_dev)
    loop2.step(0, T_dst)
    torch.cuda.synchronize()
    kd, vd = f64(loop2.kv[0].transpose(1, 2)), f64(loop2.kv[1].transpose(1, 2))
    check_tree(D, loop2.out, loop2.lse, f64(loop2.q), k2, v2, kd, vd, m, ends)
    _grow(G, k2, v2, kd, vd, path, n, ends)
    ends = [ends[b] + int(n[b]) for b in range(3)]
    q = bf16((3, 8, 128), 7300, cuda_dev)
    out, lse = torch.zeros_like(q), torch.zeros(3, 8, device=cuda_dev)
    ws = torch.zeros(int(Ld.workspace_bytes), dtype=torch.uint8, device=cuda_dev)
    kvq.decode_attention_ragged(Ld, dst, q, loop2.len[1], 260, out, SCALE, lse, ws)
    torch.cuda.synchronize()
    none = np.zeros((3, 4, 1, 128))
    ref, lr = tree_reference(D, f64(q)[:, None], k2, v2, none, none, np.zeros((1, 1), np.uint64), ends)
    vmax = np.repeat(np.abs(v2).max(axis=(2, 3)), 2, axis=1)[:, :, None]
    assert np.all(np.abs(f64(out) - ref[:, 0]) <= 4e-3 * vmax)
    assert np.abs(f64(lse) - lr[:, 0]).max() <= 2e-3


def test_steps_captured_and_replayed(cuda_dev, kvq):
    """Two steps captured in one graph (lengths in turn), replayed with new
    inputs: the same bits as eager calls."""
    c = Case(2, 6, 2, 400, 10, 300, 8, 4, 32, [1])
    n_q, max_path, T = 7, 4, 360
    A, E = Filled(c, 7400, cuda_dev), Filled(c, 7400, cuda_dev)
    ga, ea = Loop(A, n_q, max_path, [310, 333], cuda_dev), Loop(E, n_q, max_path, [310, 333], cuda_dev)
    ga.fill(7500, cuda_dev)
    ea.fill(7500, cuda_dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ga.step(0, T)   # the first calls set kernel attributes
        ga.step(1, T)
    torch.cuda.current_stream().wait_stream(s)
    ea.step(0, T)
    ea.step(1, T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ga.step(0, T)
        ga.step(1, T)
    for r in range(3):
        ga.fill(7600 + r, cuda_dev)
        ea.fill(7600 + r, cuda_dev)
        graph.replay()
        ea.step(0, T)
        ea.step(1, T)
        torch.cuda.synchronize()
        assert torch.equal(ga.out.view(torch.int16), ea.out.view(torch.int16))
        assert torch.equal(ga.lse, ea.lse) and torch.equal(ga.mass, ea.mass) and torch.equal(A.cache, E.cache)
        assert ga.len[0].tolist() == ea.len[0].tolist()


def test_two_streams_with_their_own_workspaces(cuda_dev, kvq):
    """Tree calls in flight at once on two streams, and mass and eviction
    beside them: each equals its own call alone."""
    c = Case(2, 8, 4, 3000, 10, 2900, 4, 2, 64, [0])
    F = Filled(c, 7700, cuda_dev)
    n_q, T = 16, 2950
    mask = masks_to(cuda_dev, random_tree(n_q, 1, 3))
    sets = []
    for k in range(2):
        q, x = bf16((2, n_q, 8, 128), 7710 + k, cuda_dev), bf16((2, 2, n_q, 4, 128), 7720 + k, cuda_dev)
        sets.append((q, x[0].transpose(1, 2), x[1].transpose(1, 2), torch.zeros_like(q), torch.zeros(2, n_q, 8, device=cuda_dev),
                     torch.zeros(kvq.decode_tree_workspace_bytes(F.L, n_q), dtype=torch.uint8, device=cuda_dev),
                     torch.zeros(2, 4, 3000, device=cuda_dev)))
    D = Case(2, 8, 4, 1100, 10, 1010, 4, 2, 64, [0]).layout()

    def work(k, stream=None):
        q, kd, vd, out, lse, ws, mass = sets[k]
        kvq.decode_attention_tree(F.L, F.cache, q, kd, vd, mask, T, out, SCALE, lse, ws, stream=stream)
        kvq.attention_mass(F.L, F.cache, q, lse, T, mass, None, SCALE, stream=stream)
        dst = torch.zeros(int(D.total_bytes), dtype=torch.uint8, device=cuda_dev)
        keep = torch.zeros(2, 4, 1040, dtype=torch.int32, device=cuda_dev)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        kvq.cache_evict(F.L, F.cache, mass, T, D, dst, 1040, keep, 10, stream=stream)
        return [t.clone() for t in (out, lse, mass)] if stream is None else (dst, keep)

    alone, kept = [], []
    for k in range(2):
        alone.append(work(k))
        torch.cuda.synchronize()
    want = []
    for k in range(2):
        want.append([t.clone() for t in sets[k][3:5]] + [sets[k][6].clone()])
        for t in (sets[k][3], sets[k][4], sets[k][6]):
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for r in range(4):
        kept.append([work(k, streams[k]) for k in range(2)])
    torch.cuda.synchronize()
    for k in range(2):
        for got, ref in zip((sets[k][3], sets[k][4], sets[k][6]), want[k]):
            assert torch.equal(got, ref)
        for r in range(1, 4):
            assert torch.equal(kept[r][k][0], kept[0][k][0]) and torch.equal(kept[r][k][1], kept[0][k][1])


def test_commit_is_seen_by_an_early_copying_decode(cuda_dev, kvq):
    """With kvq_set_cache_preload a decode call copies cache rows before the
    previous kernel has finished: committed and evicted rows are there."""
    c = Case(1, 28, 4, 1000, 14, 900, 4, 2, 64, [0])
    F = Filled(c, 7800, cuda_dev)
    n_q, T = 8, 950
    x = bf16((2, 1, n_q, 4, 128), 7801, cuda_dev)
    kd, vd = x[0].transpose(1, 2), x[1].transpose(1, 2)
    q = bf16((1, 28, 128), 7802, cuda_dev)
    path = torch.arange(n_q, dtype=torch.int32, device=cuda_dev)[None].contiguous()
    cnt = torch.full((1,), n_q, dtype=torch.int32, device=cuda_dev)
    ws = torch.zeros(int(F.L.workspace_bytes), dtype=torch.uint8, device=cuda_dev)
    out = [torch.zeros_like(q) for _ in range(2)]
    zero = torch.zeros_like(kd.contiguous())
    try:
        for r in range(20):
            for k, early in enumerate((False, True)):
                kvq.set_cache_preload(early)
                kvq.quantize_append(F.L, F.cache, zero, zero, T)  # so that a missed commit would show
                kvq.tree_commit(F.L, F.cache, kd, vd, path, cnt, T)
                kvq.decode_attention(F.L, F.cache, q, T + n_q, out[k], SCALE, None, ws)
            torch.cuda.synchronize()
            assert torch.equal(out[0], out[1])
    finally:
        kvq.set_cache_preload(False)


def test_waits_that_give_up(cuda_dev, kvq):
    """With a limit of one poll a tree call either completes or marks its
    workspace and leaves NaN rows; the next call is right again."""
    c = Case(2, 8, 2, 2000, 10, 1900, 4, 2, 64, [0])
    F = Filled(c, 7900, cuda_dev)
    n_q, T = 12, 1950
    q, x = bf16((2, n_q, 8, 128), 7901, cuda_dev), bf16((2, 2, n_q, 2, 128), 7902, cuda_dev)
    kd, vd = x[0].transpose(1, 2), x[1].transpose(1, 2)
    m = random_tree(n_q, 1, 5)
    mask = masks_to(cuda_dev, m)
    out, lse = torch.zeros_like(q), torch.zeros(2, n_q, 8, device=cuda_dev)
    ws = torch.zeros(kvq.decode_tree_workspace_bytes(F.L, n_q), dtype=torch.uint8, device=cuda_dev)
    try:
        kvq.set_wait_limits(1, 0)
        kvq.decode_attention_tree(F.L, F.cache, q, kd, vd, mask, T, out, SCALE, lse, ws)
        torch.cuda.synchronize()
    finally:
        kvq.set_wait_limits(0, 0)
    if kvq.workspace_status(ws):
        assert kvq.workspace_status(ws) == kvq.STATUS_TILE_WAIT
        assert torch.isnan(out.float()).any() and torch.isnan(lse).any()
    ws.zero_()
    kvq.decode_attention_tree(F.L, F.cache, q, kd, vd, mask, T, out, SCALE, lse, ws)
    torch.cuda.synchronize()
    assert kvq.workspace_status(ws) == 0
    check_tree(c, out, lse, f64(q), F.khat, F.vhat, f64(kd), f64(vd), m, [T, T])
