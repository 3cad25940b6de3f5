"""A chain of drafted tokens, and the one token behind a path, decoded with
kvq_decode_attention_window where the lengths are on the device: the rotated rows are
placed by kvq_tree_commit with the path 0, 1, 2, .., then attended."""
import numpy as np
import pytest
import torch

from gpu_helpers import Case
from serving_ref import Filled, bf16, f64
from step_ref import check_rope, check_window

pytestmark = pytest.mark.gpu
AXES = [0] * 16 + [1] * 24 + [2] * 24


@pytest.mark.parametrize("n", [1, 5, 33])
@pytest.mark.parametrize("captured", [False, True])
def test_chain_is_placed_and_attended(cuda_dev, kvq, n, captured):
    c = Case(3, 8, 4, 500, 12, 400, 4, 2, 64, [0], konly=[2])
    F = Filled(c, 9000, cuda_dev)
    khat, vhat, lens = F.khat.copy(), F.vhat.copy(), [410, 403, 460]
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device=cuda_dev)  # noqa: E731
    old, new = torch.tensor(lens, dtype=torch.int32, device=cuda_dev), z(3)
    path = torch.arange(n, dtype=torch.int32, device=cuda_dev).expand(3, n).contiguous()
    count = torch.full((3,), n, dtype=torch.int32, device=cuda_dev)
    src = bf16((3, n, 16, 128), 9001, cuda_dev)
    qkv, q, out, lse = src.clone(), z(3, n, 8, 128, t=torch.bfloat16), z(3, n, 8, 128, t=torch.bfloat16), z(3, n, 8, t=torch.float32)
    pos = (old[:, None] + torch.arange(n, device=cuda_dev)).int()[None].expand(3, 3, n).contiguous()
    freq = torch.from_numpy((1e6 ** (-np.arange(64) / 64.0)).astype(np.float32)).to(cuda_dev)
    R = kvq.rope_desc(128, AXES)

    def step():
        k, v = qkv[:, :, 8:12], qkv[:, :, 12:]
        kvq.norm_rope(F.L, R, qkv[:, :, :8], k, pos, freq, q, k)
        kvq.tree_commit(F.L, F.cache, k.transpose(1, 2), v.transpose(1, 2), path, count, 460, seq_len=old, new_len=new)
        kvq.decode_attention_window(F.L, F.cache, q, c.T_cap, 20, 150, out, None, lse, seq_len=new)

    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        g.replay()
    else:
        step()
    torch.cuda.synchronize()
    assert new.tolist() == [x + n for x in lens]
    rows = f64(qkv[:, :, 8:12])
    check_rope(qkv[:, :, 8:12], f64(src[:, :, 8:12]), pos.cpu().numpy(), f64(freq), AXES, 128, False, None, 0.0)
    for b in range(3):
        khat[b, :, lens[b]:lens[b] + n], vhat[b, :, lens[b]:lens[b] + n] = np.swapaxes(rows[b], 0, 1), np.swapaxes(f64(src[b, :, 12:]), 0, 1)
    check_window(c, out, lse, f64(q), khat, vhat, [x + n for x in lens], 20, 150)
