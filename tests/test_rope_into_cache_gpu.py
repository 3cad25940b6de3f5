"""kvq_norm_rope writing K rows where they stay, into the text rows of a cache,
with a decode behind it that copies its first cache tiles early."""
import numpy as np
import pytest
import torch

from gpu_helpers import Case
from serving_ref import SCALE, Filled, bf16

pytestmark = pytest.mark.gpu


def text_rows(L, cache, segment):
    """[B, H_kv, T_text, D] view of the text rows."""
    d, o = L.d, int(L.off[segment])
    return cache[o:o + d.B * d.H_kv * int(L.T_text) * 256].view(torch.bfloat16).view(d.B, d.H_kv, int(L.T_text), 128)


@pytest.mark.parametrize("B,vs,ve,T", [(1, 14, 100, 990), (1, 0, 0, 300), (2, 14, 600, 900), (1, 900, 950, 960)])
@pytest.mark.parametrize("call", ["decode_attention", "decode_step", "window between"])
def test_rotated_rows_are_in_early_copies(cuda_dev, kvq, B, vs, ve, T, call):
    c = Case(B, 28, 4, 1000, vs, ve, 4, 2, 64, [0])
    F = Filled(c, 8800, cuda_dev)
    L, n = F.L, T - (ve - vs)  # every text row below T
    k_out = text_rows(L, F.cache, kvq.SEG_TEXT_K)[:, :, :n].transpose(1, 2)
    ks = [bf16((B, n, 4, 128), 8801 + i, cuda_dev) for i in range(2)]
    pos = torch.arange(n, dtype=torch.int32, device=cuda_dev)[None].expand(3, n).contiguous()
    freq = torch.from_numpy((1e6 ** (-np.arange(64) / 64.0)).astype(np.float32)).to(cuda_dev)
    w = 1 + 0.25 * bf16((128,), 8805, cuda_dev)
    R = kvq.rope_desc(128, [0] * 16 + [1] * 24 + [2] * 24)
    q, new = bf16((B, 28, 128), 8806, cuda_dev), bf16((2, B, 4, 128), 8807, cuda_dev)
    ws = torch.zeros(int(L.workspace_bytes), dtype=torch.uint8, device=cuda_dev)
    other, out = torch.empty_like(q), [torch.zeros_like(q) for _ in range(3)]

    def chain(k, to, wait):
        kvq.norm_rope(L, R, None, k, pos, freq, None, k_out, None, w)
        if wait:
            torch.cuda.synchronize()
        if call == "window between":
            kvq.decode_attention_window(L, F.cache, q, T, 4, 64, other)
        if call == "decode_step":
            kvq.decode_step(L, F.cache, q, new[0], new[1], T, to, SCALE, None, ws)
        else:
            kvq.decode_attention(L, F.cache, q, T, to, SCALE, None, ws)

    for i in range(2):
        chain(ks[i], out[i], True)
    torch.cuda.synchronize()
    assert not torch.equal(out[0], out[1])
    try:
        kvq.set_cache_preload(True)
        for r in range(20):
            chain(ks[r % 2], out[2], False)
            torch.cuda.synchronize()
            assert torch.equal(out[2], out[r % 2])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain(ks[0], out[2], False)
            chain(ks[1], out[2], False)
        for r in range(5):
            out[2].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[2], out[1])
    finally:
        kvq.set_cache_preload(False)
