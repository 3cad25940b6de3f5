"""A decode step as a serving loop runs it: the drafted rows normed and rotated,
tree attention, verification, the commit of the accepted path, and windowed
decode on the new lengths -- several steps on device lengths, captured and
replayed, on two streams, behind appended rows, with waits that give up."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import bit_mixed_precision_kvq_gb300 as kvq
from gpu_helpers import Case
from serving_ref import SCALE, Filled, bf16, check_tree, f64, masks_to
from step_ref import check_rope, check_verify, check_window, parents_of, verify_reference

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
AXES = [0] * 16 + [1] * 24 + [2] * 24


def rooted_tree(n, rows, seed, reach=4):
    g = np.random.default_rng(seed)
    m = np.ones((rows, n), np.uint64)
    for b in range(rows):
        for j in range(1, n):
            m[b, j] = m[b, int(g.integers(max(0, j - reach), j))] | np.uint64(1 << j)
    return m


class Step:
    """Buffers of a loop that drafts n_q tokens a step over a vocabulary of V."""

    def __init__(self, F, n_q, V, lens, dev):
        c = F.c
        self.F, self.n_q, self.V, self.dev = F, n_q, V, dev
        H = c.H_q + 2 * c.H_kv
        z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=dev)  # noqa: E731
        self.qkv, self.q, self.out = z(c.B, n_q, H, 128), z(c.B, n_q, c.H_q, 128), z(c.B, n_q, c.H_q, 128)
        self.pos, self.mask = z(3, c.B, n_q, t=torch.int32), z(c.B, n_q, t=torch.int64)
        self.freq = torch.from_numpy((1e6 ** (-np.arange(64) / 64.0)).astype(np.float32)).to(dev)
        self.wq, self.wk = 1 + 0.25 * bf16((128,), 1, dev), 1 + 0.25 * bf16((128,), 2, dev)
        self.logits, self.tokens = z(c.B, n_q, V, t=torch.float32), z(c.B, n_q, t=torch.int32)
        self.u, self.race, self.size = z(c.B, n_q, t=torch.float32), z(c.B, V, t=torch.float32), z(c.B, t=torch.int32)
        self.lse, self.logp = z(c.B, n_q, c.H_q, t=torch.float32), z(c.B, n_q, t=torch.float32)
        self.path, self.count, self.token = z(c.B, n_q, t=torch.int32), z(c.B, t=torch.int32), z(c.B, t=torch.int32)
        self.len = [torch.tensor(lens, dtype=torch.int32, device=dev), z(c.B, t=torch.int32)]
        self.q1, self.out1, self.lse1 = z(c.B, c.H_q, 128), z(c.B, c.H_q, 128), z(c.B, c.H_q, t=torch.float32)
        self.ws = z(kvq.decode_tree_workspace_bytes(F.L, n_q), t=torch.uint8)
        self.R = kvq.rope_desc(128, AXES)

    def fill(self, seed, lens, sizes=None):
        c, n, V = self.F.c, self.n_q, self.V
        g = np.random.default_rng(seed)
        self.h = h = dict(m=rooted_tree(n, c.B, seed), tokens=g.integers(0, V, (c.B, n)).astype(np.int32), u=g.random((c.B, n)).astype(np.float32),
                          race=g.exponential(size=(c.B, V)).astype(np.float32), x=g.normal(0, 2, (c.B, n, V)).astype(np.float32),
                          size=np.array(sizes or [n] * c.B, np.int32), pos=np.zeros((3, c.B, n), np.int32))
        par = parents_of(h["m"])
        for b in range(c.B):
            for j in range(n):
                depth = bin(int(h["m"][b, j])).count("1") - 1
                h["pos"][:, b, j] = max(0, lens[b] or 0) + depth + np.array([0, j % 3, 2 * j])
                if j:  # the parent's row likes this token
                    h["x"][b, par[b, j], h["tokens"][b, j]] += 9
        self.h["qkv"] = bf16(self.qkv.shape, seed, self.dev)
        self.qkv.copy_(self.h["qkv"])
        self.q1.copy_(bf16(self.q1.shape, seed + 1, self.dev))
        for to, name in ((self.tokens, "tokens"), (self.u, "u"), (self.race, "race"), (self.logits, "x"), (self.size, "size"), (self.pos, "pos")):
            to.copy_(torch.from_numpy(h[name]).to(self.dev))
        self.mask.copy_(masks_to(self.dev, h["m"]))

    def parts(self):
        c = self.F.c
        q, k, v = self.qkv[:, :, :c.H_q], self.qkv[:, :, c.H_q:c.H_q + c.H_kv], self.qkv[:, :, c.H_q + c.H_kv:]
        return q, k, v

    def step(self, k, T, stream=None):
        """One step from the lengths len[k] to len[1 - k]; T: the longest context."""
        F, old, new = self.F, self.len[k], self.len[1 - k]
        q, kd, vd = self.parts()
        kvq.norm_rope(F.L, self.R, q, kd, self.pos, self.freq, self.q, kd, self.wq, self.wk, stream=stream)  # K where it lies
        kt, vt = kd.transpose(1, 2), vd.transpose(1, 2)
        kvq.decode_attention_tree(F.L, F.cache, self.q, kt, vt, self.mask, T, self.out, SCALE, self.lse, self.ws, seq_len=old, stream=stream)
        kvq.tree_verify(self.logits, self.tokens, self.mask, self.u, self.race, self.path, self.count, self.token, tree_len=self.size,
                        logprob=self.logp, stream=stream)
        kvq.tree_commit(F.L, F.cache, kt, vt, self.path, self.count, T, seq_len=old, new_len=new, stream=stream)
        kvq.decode_attention_window(F.L, F.cache, self.q1, F.c.T_cap, 20, 150, self.out1, SCALE, self.lse1, seq_len=new, stream=stream)

    def results(self):
        return [self.q, self.qkv, self.out, self.lse, self.path, self.count, self.token, self.logp, self.len[0], self.len[1], self.out1, self.lse1,
                self.F.cache]


def test_steps_match_references(cuda_dev, kvq):
    """Three steps; in the second a sequence's tree is empty, and it is inactive from there on."""
    c = Case(3, 8, 4, 500, 12, 400, 4, 2, 64, [0], konly=[2])
    F = Filled(c, 8000, cuda_dev)
    khat, vhat = F.khat.copy(), F.vhat.copy()
    lens, n_q, V, T = [420, 405, 460], 9, 5003, 490
    s = Step(F, n_q, V, lens, cuda_dev)
    for r in range(3):
        s.fill(8100 + 10 * r, lens, [n_q, n_q if r != 1 else 0, 5])
        s.step(r % 2, T)
        torch.cuda.synchronize()
        h = s.h
        q, k, v = (f64(h["qkv"][:, :, a:b]) for a, b in ((0, 8), (8, 12), (12, 16)))
        freq = f64(s.freq)
        check_rope(s.q, q, h["pos"], freq, AXES, 128, False, f64(s.wq), 1e-6)
        check_rope(s.parts()[1], k, h["pos"], freq, AXES, 128, False, f64(s.wk), 1e-6)
        kd, vd = f64(s.parts()[1].transpose(1, 2)), f64(s.parts()[2].transpose(1, 2))
        assert np.array_equal(vd, np.swapaxes(v, 1, 2))
        check_tree(c, s.out, s.lse, f64(s.q), khat, vhat, kd, vd, h["m"], lens)
        check_verify((s.path, s.count, s.token, s.logp), verify_reference(h["x"], h["tokens"], h["m"], h["u"], h["race"], None, None, h["size"]))
        path, n = s.path.cpu().numpy(), s.count.cpu().numpy()
        for b in range(3):
            if lens[b] is None or n[b] < 0:
                lens[b] = None
                continue
            for i in range(n[b]):
                khat[b, :, lens[b] + i], vhat[b, :, lens[b] + i] = kd[b, :, path[b, i]], vd[b, :, path[b, i]]
            lens[b] += int(n[b])
        assert s.len[1 - r % 2].tolist() == [-1 if x is None else x for x in lens]
        check_window(c, s.out1[:, None], s.lse1[:, None], f64(s.q1)[:, None], khat, vhat, lens, 20, 150)
    assert lens[1] is None and sum(x is None for x in lens) == 1


def test_steps_captured_and_replayed(cuda_dev, kvq):
    """Two steps captured in one graph, replayed with new inputs: the bits of eager calls."""
    c = Case(2, 6, 2, 600, 10, 300, 8, 4, 32, [1])
    n_q, V, T = 7, 3001, 560
    sets = [Step(Filled(c, 8200, cuda_dev), n_q, V, [310, 333], cuda_dev) for _ in range(2)]
    for s in sets:
        s.fill(8210, [310, 333])
        s.step(0, T)
        s.step(1, T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sets[0].step(0, T)
        sets[0].step(1, T)
    for r in range(4):
        for s in sets:
            s.fill(8300 + r, [310, 333])
        graph.replay()
        sets[1].step(0, T)
        sets[1].step(1, T)
        torch.cuda.synchronize()
        for a, b in zip(sets[0].results(), sets[1].results()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # five rounds of two steps, each storing its tree's token 0 at least
    assert sets[0].len[0][0] >= 310 + 10 and sets[0].len[0][1] >= 333 + 10


def test_steps_on_two_streams(cuda_dev, kvq):
    """Two loops in flight at once: each as alone."""
    c = Case(2, 8, 4, 3000, 10, 2900, 4, 2, 64, [0])
    want, loops = [], []
    for k in range(2):
        s = Step(Filled(c, 8400 + k, cuda_dev), 12, 20011, [2910, 2930], cuda_dev)
        s.fill(8410 + k, [2910, 2930])
        start = s.F.cache.clone()
        s.step(0, 2980)
        torch.cuda.synchronize()
        want.append([x.clone() for x in s.results()])
        loops.append((s, start))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for r in range(4):
        for s, start in loops:
            s.F.cache.copy_(start)
            s.qkv.copy_(s.h["qkv"])
            for x in s.results():
                if x is not s.F.cache and x is not s.qkv and x is not s.len[0]:
                    x.zero_()
        torch.cuda.synchronize()
        for (s, _), st in zip(loops, streams):
            s.step(0, 2980, st)
        torch.cuda.synchronize()
        for (s, _), w in zip(loops, want):
            for a, b in zip(s.results(), w):
                assert torch.equal(a, b)


def test_window_sees_what_was_written_before(cuda_dev, kvq):
    """No wait between a writer and the windowed decode behind it, with early
    copies allowed: appended and committed rows are there."""
    c = Case(1, 28, 4, 1000, 14, 900, 4, 2, 64, [0])
    F = Filled(c, 8500, cuda_dev)
    x = bf16((2, 1, 6, 4, 128), 8501, cuda_dev)
    kd, vd = x[0].transpose(1, 2), x[1].transpose(1, 2)
    zero = torch.zeros_like(kd.contiguous())
    q = bf16((1, 28, 128), 8502, cuda_dev)
    path, cnt = torch.arange(6, dtype=torch.int32, device=cuda_dev)[None].contiguous(), torch.full((1,), 6, dtype=torch.int32, device=cuda_dev)
    out = [torch.zeros_like(q) for _ in range(3)]
    kvq.quantize_append(F.L, F.cache, zero, zero, 950)
    kvq.decode_attention_window(F.L, F.cache, q, 956, 4, 40, out[0])
    kvq.tree_commit(F.L, F.cache, kd, vd, path, cnt, 950)
    torch.cuda.synchronize()
    kvq.decode_attention_window(F.L, F.cache, q, 956, 4, 40, out[1])
    torch.cuda.synchronize()
    assert not torch.equal(out[0], out[1])
    try:
        kvq.set_cache_preload(True)
        for _ in range(20):
            kvq.quantize_append(F.L, F.cache, zero, zero, 950)
            kvq.decode_attention_window(F.L, F.cache, q, 956, 4, 40, out[2])
            torch.cuda.synchronize()
            assert torch.equal(out[2], out[0])
            kvq.quantize_append(F.L, F.cache, zero, zero, 950)
            kvq.tree_commit(F.L, F.cache, kd, vd, path, cnt, 950)
            kvq.decode_attention_window(F.L, F.cache, q, 956, 4, 40, out[2])
            torch.cuda.synchronize()
            assert torch.equal(out[2], out[1])
    finally:
        kvq.set_cache_preload(False)


def test_early_copies_behind_the_new_calls(cuda_dev, kvq):
    """A decode step that copies cache rows early, behind the norm-and-rotation,
    verification and windowed calls that follow an append: none of them lets it
    start before the appended rows are there."""
    c = Case(1, 28, 4, 1000, 14, 900, 4, 2, 64, [0])
    F = Filled(c, 8600, cuda_dev)
    s = Step(F, 5, 4001, [950], cuda_dev)
    s.fill(8601, [950])
    rows = bf16((2, 1, 4, 900 - 14, 128), 8602, cuda_dev)
    zero = torch.zeros_like(rows[0])
    q = bf16((1, 28, 128), 8603, cuda_dev)
    ws = torch.zeros(int(F.L.workspace_bytes), dtype=torch.uint8, device=cuda_dev)
    out = [torch.zeros_like(q) for _ in range(2)]
    a, b, _ = s.parts()
    between = [lambda: kvq.norm_rope(F.L, s.R, a, b, s.pos, s.freq, s.q, b),
               lambda: kvq.tree_verify(s.logits, s.tokens, s.mask, s.u, s.race, s.path, s.count, s.token),
               lambda: kvq.decode_attention_window(F.L, F.cache, s.q1, 950, 4, 40, s.out1)]
    try:
        for r in range(6):
            for call in between:
                for k, early in enumerate((False, True)):
                    kvq.set_cache_preload(early)
                    kvq.quantize_append(F.L, F.cache, zero, zero, 14)
                    if not early:
                        torch.cuda.synchronize()
                    kvq.quantize_append(F.L, F.cache, rows[0], rows[1], 14)
                    call()
                    kvq.decode_attention(F.L, F.cache, q, 950, out[k], SCALE, None, ws)
                torch.cuda.synchronize()
                assert torch.equal(out[0], out[1])
    finally:
        kvq.set_cache_preload(False)


def test_verify_waits_that_give_up(cuda_dev, kvq):
    """With a limit of one poll a sequence is either right or inactive; the next
    call is right again."""
    c = Case(4, 4, 1, 64, 0, 0, 4, 4, 32, [])
    F = type("F", (), dict(c=c, L=c.layout(), cache=None))
    s = Step(F, 9, 150001, [10] * 4, cuda_dev)
    s.fill(8700, [10] * 4)

    def call():
        kvq.tree_verify(s.logits, s.tokens, s.mask, s.u, s.race, s.path, s.count, s.token, logprob=s.logp)
        torch.cuda.synchronize()
        return [x.clone() for x in (s.path, s.count, s.token, s.logp)]

    want = call()
    check_verify(want, verify_reference(s.h["x"], s.h["tokens"], s.h["m"], s.h["u"], s.h["race"]))
    try:
        kvq.set_wait_limits(1, 0)
        for _ in range(5):
            got = call()
            for b in range(4):
                if got[1][b] == -1:
                    assert (got[0][b] == -1).all() and got[2][b] == -1 and not got[3][b].any()
                else:
                    assert all(torch.equal(x[b], y[b]) for x, y in zip(got, want))
    finally:
        kvq.set_wait_limits(0, 0)
    assert all(torch.equal(x, y) for x, y in zip(call(), want))


FIRST = """
import sys
sys.path[:0] = [%r, %r]
import torch
from gpu_helpers import Case
from serving_ref import Filled
from test_step_flow_gpu import Step
dev = "cuda"
c = Case(2, 8, 2, 700, 10, 600, 4, 2, 64, [1])
sets = []
for _ in range(2):
    F = Filled(c, 9, dev)
    s = Step(F, 6, 3001, [620, 640], dev)
    s.fill(10, [620, 640])
    sets.append(s)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    sets[0].step(0, 690)
g.replay()
sets[1].step(0, 690)
torch.cuda.synchronize()
for a, b in zip(sets[0].results(), sets[1].results()):
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
assert (sets[0].len[1] > sets[0].len[0]).all() and sets[0].out1.any()
print("same")
"""


def test_first_calls_of_a_process_are_captured(cuda_dev, kvq):
    """Kernels loaded and their attributes set while a stream is captured."""
    r = subprocess.run([sys.executable, "-c", FIRST % (ROOT, os.path.join(ROOT, "tests"))], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
