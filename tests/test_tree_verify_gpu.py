"""kvq_tree_verify against the walk in 64 bits: deterministic and sampled
drafts, greedy sequences, unequal trees, odd vocabularies and strides, the rows
that end a walk, and the distribution of what it picks."""
import numpy as np
import pytest
import torch

from serving_ref import masks_to
from step_ref import check_verify, parents_of, verify_reference

pytestmark = pytest.mark.gpu


def _tree(n, rows, seed, reach=6):
    g = np.random.default_rng(seed)
    m = np.ones((rows, n), np.uint64)
    for r in range(rows):
        for j in range(1, n):
            m[r, j] = m[r, int(g.integers(max(0, j - reach), j))] | np.uint64(1 << j)
    return m


class Tree:
    """Seeded inputs: logits with a likely token a row, drafts that often hit it."""

    def __init__(self, B, n, V, half, probs, seed, shared=False):
        g = np.random.default_rng(seed)
        self.masks = _tree(n, 1 if shared else B, seed)
        x = g.normal(0, 2.5, (B, n, V)).astype(np.float32)
        hot = g.integers(0, V, (B, n))
        np.put_along_axis(x, hot[..., None], (np.log(V) + 3 + 1.5 * g.normal(size=(B, n, 1))).astype(np.float32), 2)
        self.t = torch.from_numpy(x)
        if half:
            self.t = self.t.bfloat16()
        self.x = self.t.float().numpy()
        y = x + 0.5 * g.normal(size=x.shape).astype(np.float32)
        self.draft = None
        par, self.tokens = parents_of(self.masks), np.zeros((B, n), np.int32)
        if probs:
            e = np.exp(y - y.max(-1, keepdims=True))
            self.draft = (e / e.sum(-1, keepdims=True)).astype(np.float32)
        order = np.argsort(-y, -1)[..., :n]
        for b in range(B):
            seen = {}
            for j in range(1, n):
                p = par[b % len(self.masks), j]
                if probs:
                    d = self.draft[b, p].astype(np.float64)
                    self.tokens[b, j] = g.choice(V, p=d / d.sum())
                else:
                    self.tokens[b, j] = order[b, p, min(seen.get(p, 0), order.shape[-1] - 1)]
                    seen[p] = seen.get(p, 0) + 1
        self.u = g.random((B, n)).astype(np.float32)
        self.race = g.exponential(size=(B, V)).astype(np.float32)


def run(kvq, dev, s, heat=None, size=None, logits=None, draft=None, want_logp=True):
    B, n, V = s.x.shape
    to = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    path, plen, nxt = (torch.full(sh, 77, dtype=torch.int32, device=dev) for sh in ((B, n), (B,), (B,)))
    logp = torch.full((B, n), 77.0, device=dev) if want_logp else None
    kvq.tree_verify(s.t.to(dev) if logits is None else logits, to(s.tokens), masks_to(dev, s.masks), to(s.u), to(s.race), path, plen, nxt,
                    to(s.draft) if draft is None else draft, to(None if heat is None else np.asarray(heat, np.float32)),
                    to(None if size is None else np.asarray(size, np.int32)), logp)
    return path, plen, nxt, logp


CASES = [
    # B, n_q, V, bf16, sampled, one tree
    (1, 1, 1, True, False, False), (1, 5, 2, False, True, False), (2, 4, 7, True, False, True), (3, 9, 129, False, True, False),
    (4, 26, 1000, True, False, False), (4, 26, 1001, True, True, False), (2, 64, 4099, False, False, True), (2, 64, 4099, False, True, True),
    (9, 16, 8192, True, True, False), (1, 16, 70001, True, True, False), (1, 16, 152000, True, False, False), (20, 7, 9001, False, False, False),
    (80, 3, 20000, True, False, True), (160, 3, 600, False, True, True),
    # two CTAs and one a sequence, several groups a thread, rows at every alignment
    (1, 2, 1048577, True, True, False), (77, 1, 256000, False, False, False), (50, 5, 30001, True, True, False), (80, 4, 20003, False, True, False), (40, 3, 33333, True, False, True),
]


@pytest.mark.parametrize("ci", range(len(CASES)))
def test_verify_matches_walk(cuda_dev, kvq, ci):
    B, n, V, half, probs, shared = CASES[ci]
    s = Tree(B, n, V, half, probs, 100 + ci, shared)
    ref = verify_reference(s.x, s.tokens, s.masks, s.u, s.race, s.draft)
    check_verify(run(kvq, cuda_dev, s), ref)


@pytest.mark.parametrize("half,probs", [(True, False), (False, True)])
def test_verify_temperatures_and_sizes(cuda_dev, kvq, half, probs):
    """Greedy, cold and hot sequences and trees of every size in one batch; an
    entry outside [1, n_q] is an inactive sequence."""
    B, n, V = 12, 11, 3001
    s = Tree(B, n, V, half, probs, 7)
    heat = [0.0, 1.0, 0.5, 2.0, -1.0, float("nan"), 0.25, 1.0, 1.0, 1.0, 0.0, 0.7]
    size = [11, 1, 2, 5, 11, 3, 11, 0, -4, 12, 11, 11]
    ref = verify_reference(s.x, s.tokens, s.masks, s.u, s.race, s.draft, heat, size)
    out = run(kvq, cuda_dev, s, heat, size)
    check_verify(out, ref, scores=4 * 64.0)
    for b in (7, 8, 9):
        assert out[1][b] == -1 and out[2][b] == -1 and (out[0][b] == -1).all() and (out[3][b] == 0).all()


def test_verify_greedy_ties_go_to_the_lowest(cuda_dev, kvq):
    """Equal largest logits at several places, on vector borders and across CTAs."""
    B, n, V = 4, 3, 40003
    s = Tree(B, n, V, True, False, 8)
    s.x[:] = -1.0
    at = [[5, 6, 39999], [8, 15, 16], [40002, 40001, 20000], [33, 7, 39990]]
    for b in range(B):
        s.x[b][:, at[b]] = 3.0
        s.tokens[b, 1:] = [max(at[b]), min(at[b])]
    s.masks = np.array([[1, 3, 5]], np.uint64)  # two children of token 0
    s.t = torch.from_numpy(s.x).bfloat16()
    path, plen, nxt, logp = run(kvq, cuda_dev, s, heat=[0.0] * B)
    assert path.cpu().tolist() == [[0, 2, -1]] * B and plen.tolist() == [2] * B and nxt.cpu().tolist() == [min(a) for a in at]
    check_verify((path, plen, nxt, logp), verify_reference(s.x, s.tokens, s.masks, s.u, s.race, None, [0.0] * B))


def test_verify_masked_and_broken_rows(cuda_dev, kvq):
    """-inf logits cannot be picked; NaN, +inf and rows of -inf end the sequence,
    but only where the walk meets them."""
    B, n, V = 6, 4, 5000
    s = Tree(B, n, V, False, False, 9)
    s.masks = np.array([[1, 3, 7, 15]], np.uint64)  # a chain
    s.u[:] = 0.999
    s.u[:, 1] = 0.0  # token 1 is accepted, token 2 not (its probability is below 0.999)
    s.x[0, :, 100:] = -np.inf
    s.tokens[0] = 50
    s.x[1, 0, 4321] = np.nan
    s.x[2, 1, 7] = np.inf
    s.x[3, 1, :] = -np.inf
    s.x[4, 3, :] = np.nan    # never reached
    s.x[5, :, :] = -np.inf
    s.x[5, :, 4999] = -3.0   # one token is left: p = 1
    s.tokens[5] = 4999
    s.t = torch.from_numpy(s.x)
    out = run(kvq, cuda_dev, s)
    assert out[1].cpu().tolist()[1:4] == [-1, -1, -1] and out[1][5] == 4 and out[2][5] == 4999 and 0 <= out[2][0] < 100
    check_verify(out, verify_reference(s.x, s.tokens, s.masks, s.u, s.race))


def test_verify_token_ids_outside_and_twice(cuda_dev, kvq):
    """An id outside the vocabulary is refused; a sibling with a refused one's id
    is refused too, and neither is picked afterwards."""
    B, n, V = 3, 5, 64
    s = Tree(B, n, V, True, False, 10)
    s.masks = np.array([[1, 3, 5, 9, 17]], np.uint64)  # four children of token 0
    s.tokens[0] = [0, -1, V, 2 ** 31 - 1, -2 ** 31]
    hot = int(np.argmax(s.x[1, 0]))
    s.tokens[1], s.u[1] = [0, hot, hot, hot, hot], [0, 0.9999, 0.0, 0.0, 0.0]
    s.race[1, hot] = 1e-30
    s.tokens[2], s.u[2] = [0, 3, 9, 3, 11], 0.9999
    out = run(kvq, cuda_dev, s)
    assert out[1].cpu().tolist()[:2] == [1, 1] and out[2][1] != hot
    check_verify(out, verify_reference(s.x, s.tokens, s.masks, s.u, s.race))


@pytest.mark.parametrize("probs", [False, True])
def test_verify_random_numbers_out_of_range(cuda_dev, kvq, probs):
    """What has no probability is refused whatever its random number is; a NaN
    number refuses its token.  (Numbers outside [0, 1) promise no distribution.)"""
    B, n, V = 4, 3, 100
    s = Tree(B, n, V, False, probs, 21)
    s.masks = np.array([[1, 3, 5]], np.uint64)
    s.x[:, :, 50:] = -np.inf
    s.t = torch.from_numpy(s.x)
    s.tokens[0], s.u[0] = [0, 70, -3], [0, -1.0, -5.0]    # p = 0; no such id
    s.tokens[1], s.u[1] = [0, 10, 11], np.nan
    s.tokens[2], s.u[2] = [0, 10, 11], [0, 2.0, -1.0]     # the first refused, the second taken
    if probs:
        s.draft[:, :, 10:12] = np.float32(0.01)
        s.draft[2, 0, 10] = 0.999
        s.x[2, 0, 10] = s.x[2, 0, :10].min()
        s.t = torch.from_numpy(s.x)
        s.draft[3, 0, :] = np.nan                         # everything is refused, nothing is left: r stays
    out = run(kvq, cuda_dev, s)
    assert out[1].tolist()[:3] == [1, 1, 2] and out[0][2].tolist() == [0, 2, -1]
    assert all(0 <= int(t) < 50 for t in out[2])
    if probs:
        assert out[1][3] == 1


def test_verify_race_without_entries(cuda_dev, kvq):
    """Entries of the race that are not above 0 are never picked; with none at
    all the token of the largest logit is."""
    B, n, V = 3, 1, 777
    s = Tree(B, n, V, False, False, 11)
    s.race[0, :] = 0.0
    s.race[1, 1:] = -1.0
    s.race[2, ::2] = np.nan
    out = run(kvq, cuda_dev, s)
    assert out[2][0] == int(np.argmax(s.x[0, 0])) and out[2][1] == 0 and out[2][2] % 2 == 1


@pytest.mark.parametrize("half", [True, False])
def test_verify_strided_rows(cuda_dev, kvq, half):
    """Rows at every alignment (an odd pitch), and tokens cut from a longer buffer."""
    B, n, V = 3, 8, 4001
    s = Tree(B, n, V, half, True, 12)
    wide = torch.full((B, n + 3, V + 2), float("nan"), dtype=s.t.dtype, device=cuda_dev)
    wide[:, 1:n + 1, 1:V + 1] = s.t.to(cuda_dev)
    q = torch.full((B, n + 1, V + 5), float("nan"), device=cuda_dev)
    q[:, :n, 3:V + 3] = torch.from_numpy(s.draft).to(cuda_dev)
    out = run(kvq, cuda_dev, s, logits=wide[:, 1:n + 1, 1:V + 1], draft=q[:, :n, 3:V + 3])
    check_verify(out, verify_reference(s.x, s.tokens, s.masks, s.u, s.race, s.draft))
    same = run(kvq, cuda_dev, s, want_logp=False)
    for a, b in zip(out[:3], same[:3]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("probs", [False, True])
def test_verify_draws_from_the_target(cuda_dev, kvq, probs):
    """The first token behind token 0 -- an accepted draft or the one picked --
    is distributed as the target's softmax whatever the drafts were: 40,000
    sequences over a vocabulary of 12, every count within 5.5 standard
    deviations (1e-6 for the lot by the normal tail)."""
    B, n, V = 40000, 4, 12
    g = np.random.default_rng(13)
    x = g.normal(0, 1.2, V).astype(np.float32)
    q = np.exp(g.normal(0, 1.0, V))
    q = (q / q.sum()).astype(np.float32)
    s = Tree.__new__(Tree)
    s.x = np.broadcast_to(x, (B, n, V))
    s.t = torch.from_numpy(np.ascontiguousarray(s.x))
    s.masks = np.array([[1, 3, 5, 9]], np.uint64)  # three children of token 0
    s.draft = np.ascontiguousarray(np.broadcast_to(q, (B, n, V))) if probs else None
    s.tokens = g.choice(V, (B, n), p=q / q.sum(dtype=np.float64)).astype(np.int32) if probs else np.tile(np.array([0, 3, 1, 7], np.int32), (B, 1))
    s.u, s.race = g.random((B, n)).astype(np.float32), g.exponential(size=(B, V)).astype(np.float32)
    path, plen, nxt, _ = (y.cpu().numpy() for y in run(kvq, cuda_dev, s))
    first = np.where(plen > 1, np.take_along_axis(s.tokens, np.maximum(path[:, 1:2], 0), 1)[:, 0], nxt)
    p = np.exp(x.astype(np.float64) - x.max())
    p /= p.sum()
    count = np.bincount(first, minlength=V)
    assert np.all(np.abs(count - B * p) <= 5.5 * np.sqrt(B * p * (1 - p)))


def test_verify_is_repeatable(cuda_dev, kvq):
    s = Tree(5, 20, 33333, True, True, 14)
    a, b = run(kvq, cuda_dev, s), run(kvq, cuda_dev, s)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_verify_rows_past_32_bits(cuda_dev, kvq):
    """Rows more than 2^32 bytes apart."""
    B, n, V = 2, 4, 5003
    s = Tree(B, n, V, True, True, 22)
    want = run(kvq, cuda_dev, s)
    big, far = torch.empty(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device=cuda_dev), 2 ** 31 + 8192
    logits = big.as_strided((B, n, V), (far, V + 5, 1))
    logits.copy_(s.t)
    got = run(kvq, cuda_dev, s, logits=logits)
    del logits, big
    q = torch.empty(2 ** 30 + 2 ** 20, device=cuda_dev).as_strided((B, n, V), (2 ** 30 + 4099, V, 1))
    q.copy_(torch.from_numpy(s.draft))
    again = run(kvq, cuda_dev, s, draft=q)
    # (rows at other 16-byte boundaries are summed in another order)
    ref = verify_reference(s.x, s.tokens, s.masks, s.u, s.race, s.draft)
    for out in (want, got, again):
        check_verify(out, ref)
