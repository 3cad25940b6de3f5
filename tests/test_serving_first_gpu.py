"""The serving calls where nothing of theirs has run yet."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np, torch
import bit_mixed_precision_kvq_gb300 as kvq
from gpu_helpers import Case
from serving_ref import SCALE, bf16, masks_to, random_tree
dev = "cuda"
c = Case(2, 8, 2, 700, 10, 600, 4, 2, 64, [1])
L, Ld = c.layout(), Case(2, 8, 2, 300, 10, 210, 4, 2, 64, [1]).layout()
n_q, T = 6, 650
cache = torch.randint(0, 60, (int(L.total_bytes),), dtype=torch.uint8, device=dev)
q, x = bf16((2, n_q, 8, 128), 1, dev), bf16((2, 2, n_q, 2, 128), 2, dev)
kd, vd = x[0].transpose(1, 2), x[1].transpose(1, 2)
mask = masks_to(dev, random_tree(n_q, 2, 3))
path = torch.arange(4, dtype=torch.int32, device=dev).repeat(2, 1)
cnt = torch.tensor([4, 2], dtype=torch.int32, device=dev)
def buffers():
    return dict(cache=cache.clone(), out=torch.zeros_like(q), lse=torch.zeros(2, n_q, 8, device=dev), new=torch.zeros(2, dtype=torch.int32, device=dev),
        mass=torch.zeros(2, 2, 700, device=dev), dst=torch.zeros(int(Ld.total_bytes), dtype=torch.uint8, device=dev),
        keep=torch.zeros(2, 2, 240, dtype=torch.int32, device=dev), ws=torch.zeros(kvq.decode_tree_workspace_bytes(L, n_q), dtype=torch.uint8, device=dev))
def work(s):
    kvq.decode_attention_tree(L, s["cache"], q, kd, vd, mask, T, s["out"], SCALE, s["lse"], s["ws"])
    kvq.tree_commit(L, s["cache"], kd, vd, path, cnt, T, new_len=s["new"])
    kvq.attention_mass(L, s["cache"], q, s["lse"], T + 4, s["mass"], None, SCALE, seq_len=s["new"], path=path, path_len=cnt)
    kvq.cache_evict(L, s["cache"], s["mass"], T + 4, Ld, s["dst"], 240, s["keep"], 5, None, s["new"])
a, b = buffers(), buffers()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    work(a)
g.replay()
work(b)
torch.cuda.synchronize()
for k in a:
    if k != "ws":
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
assert a["new"].tolist() == [654, 652] and (a["keep"] >= 0).all() and float(a["mass"].sum()) > 0
print("same")
"""


def test_first_calls_of_a_process_are_captured(cuda_dev, kvq):
    """Kernels loaded and their attributes set while a stream is captured."""
    r = subprocess.run([sys.executable, "-c", FIRST % (ROOT, os.path.join(ROOT, "tests"))], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
