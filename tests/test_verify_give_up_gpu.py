"""kvq_tree_verify where its CTAs' waits for one another give up: the sequence is
right or inactive, every CTA stays until the parts that were sent to it have
come, and the calls behind it are as ever."""
import numpy as np
import pytest
import torch

from serving_ref import masks_to
from step_ref import check_verify, verify_reference

pytestmark = pytest.mark.gpu


class Walks:
    """B sequences of a chain of n tokens behind token 0; every third child is refused."""

    def __init__(self, B, n, V, probs, seed, dev):
        g = np.random.default_rng(seed)
        self.masks = np.array([[(1 << (j + 1)) - 1 for j in range(n)]], np.uint64)
        self.x = g.normal(0, 2, (B, n, V)).astype(np.float32)
        self.tokens = g.integers(0, V, (B, n)).astype(np.int32)
        self.draft = None
        for j in range(1, n):
            self.x[np.arange(B), j - 1, self.tokens[:, j]] += 14
        if probs:
            e = np.exp(self.x - self.x.max(-1, keepdims=True))
            self.draft = (e / e.sum(-1, keepdims=True) * 0.9).astype(np.float32)
        self.u = g.random((B, n)).astype(np.float32) * 0.5
        self.u[:, 3::3] = 0.99999994
        if probs:
            self.draft[:, 2::3] *= 8  # the ratio test refuses there
        self.race = g.exponential(size=(B, V)).astype(np.float32)
        to = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.ins = [to(self.x), to(self.tokens), masks_to(dev, self.masks), to(self.u), to(self.race)]
        self.q = to(self.draft)
        i32 = dict(dtype=torch.int32, device=dev)
        self.outs = [torch.full((B, n), 77, **i32), torch.full((B,), 77, **i32), torch.full((B,), 77, **i32), torch.full((B, n), 77.0, device=dev)]

    def call(self, kvq):
        kvq.tree_verify(*self.ins, *self.outs[:3], draft_prob=self.q, logprob=self.outs[3])

    def check(self, want):
        """How many sequences gave up; the others are `want`."""
        late = self.outs[1].cpu() == -1
        for b in range(len(late)):
            if late[b]:
                assert (self.outs[0][b] == -1).all() and self.outs[2][b] == -1 and not self.outs[3][b].any()
            else:
                assert all(torch.equal(x[b], y[b]) for x, y in zip(self.outs, want))
        return int(late.sum())


@pytest.mark.parametrize("B,V", [(1, 150001), (4, 150001), (9, 60000), (37, 40000), (60, 33000)])
@pytest.mark.parametrize("probs", [False, True])
def test_walks_that_give_up(cuda_dev, kvq, B, V, probs):
    """Clusters of 16, 8, 4 and 2 CTAs.  One poll without suspending finds no part
    that has to come from another CTA; a few more may or may not."""
    s = Walks(B, 8, V, probs, 100 + B, cuda_dev)
    s.call(kvq)
    want = [x.clone() for x in s.outs]
    check_verify(want, verify_reference(s.x, s.tokens, s.masks, s.u, s.race, s.draft))
    gave_up = 0
    try:
        for polls in [1, 2, 1, 3, 1, 5, 1, 1]:
            kvq.set_wait_limits(polls, 0)
            for x in s.outs:
                x.fill_(55)
            s.call(kvq)
            torch.cuda.synchronize()
            gave_up += s.check(want)
        assert gave_up >= 5 * B  # all of those with one poll
        # calls that give up back to back, in the shared memory that the last one left
        kvq.set_wait_limits(1, 0)
        for _ in range(50):
            s.call(kvq)
    finally:
        kvq.set_wait_limits(0, 0)
    for x in s.outs:
        x.fill_(55)
    s.call(kvq)
    torch.cuda.synchronize()
    assert s.check(want) == 0


def test_walks_that_give_up_while_captured(cuda_dev, kvq):
    """A captured call keeps the limit of its capture; replays before and behind
    calls with the default limit."""
    s, t = Walks(4, 8, 150001, True, 7, cuda_dev), Walks(4, 8, 150001, True, 7, cuda_dev)
    s.call(kvq)
    want = [x.clone() for x in s.outs]
    g = torch.cuda.CUDAGraph()
    try:
        kvq.set_wait_limits(1, 0)
        with torch.cuda.graph(g):
            s.call(kvq)
    finally:
        kvq.set_wait_limits(0, 0)
    for _ in range(10):
        for x in t.outs:
            x.fill_(55)
        g.replay()
        t.call(kvq)
        torch.cuda.synchronize()
        assert s.check(want) == 4 and t.check(want) == 0
