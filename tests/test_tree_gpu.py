"""kvq_decode_attention_tree and kvq_tree_commit against 64-bit references
over the oracle's reconstruction of the cache (tests/serving_ref.py has the
tolerances and where they come from)."""
import numpy as np
import pytest
import torch

import bit_mixed_precision_kvq_gb300 as kvq
import synth
from gpu_helpers import Case, bits
from serving_ref import SCALE, Filled, bf16, check_tree, f64, masks_to, random_tree

pytestmark = pytest.mark.gpu


def _call(F, q, kd, vd, masks, T, lens=None, lse=True, dev="cuda", ws=None):
    B, n_q, Hq, D = q.shape
    out = torch.full((B, n_q, Hq, D), 5.0, dtype=torch.bfloat16, device=dev)
    l = torch.full((B, n_q, Hq), 9.0, device=dev) if lse else None
    if ws is None:
        ws = torch.full((kvq.decode_tree_workspace_bytes(F.L, n_q),), 0x3C, dtype=torch.uint8, device=dev)
        ws[:4] = 0
    sl = torch.tensor(lens, dtype=torch.int32, device=dev) if lens is not None else None
    kvq.decode_attention_tree(F.L, F.cache, q, kd, vd, masks_to(dev, masks), T, out, SCALE, l, ws, seq_len=sl)
    torch.cuda.synchronize()
    assert kvq.workspace_status(ws) == 0
    return out, l


def _drafts(c, n_q, seed, dev):
    """K and V as a projection leaves them, [B, n_q, H_kv, D], seen head-first."""
    x = bf16((2, c.B, n_q, c.H_kv, c.D), seed, dev)
    return x[0].transpose(1, 2), x[1].transpose(1, 2)


def _active(lens, T):
    return [n if 0 <= n <= T else None for n in lens]


CASES = [
    # layout, n_q, T_ctx, lengths (None: uniform)
    (Case(1, 4, 1, 300, 14, 256, 4, 4, 32, []), 5, 257, None),                    # g = 4, odd everything
    (Case(1, 28, 4, 700, 14, 640, 4, 2, 64, [0]), 16, 690, None),                 # g = 7: 112 columns
    (Case(2, 8, 8, 300, 10, 250, 8, 4, 32, [1], konly=[2]), 8, 300, None),        # one query head per KV head
    (Case(2, 32, 8, 500, 32, 400, 2, 2, 32, [3]), 3, 480, None),
    (Case(1, 4, 4, 400, 16, 300, 2, 4, 128, [0]), 64, 400, None),                 # 64 tokens: bit 63
    (Case(3, 6, 2, 300, 0, 290, 16, 16, 64, [], konly=[1]), 7, 295, None),        # unquantised, no prefix
    (Case(2, 5, 1, 300, 8, 8, 4, 4, 64, []), 9, 200, None),                       # no visual block
    (Case(2, 8, 2, 900, 20, 800, 8, 8, 128, []), 33, 860, [860, 411]),            # cut inside the visual block
    (Case(5, 8, 2, 300, 16, 272, 4, 2, 64, [1]), 6, 290, [0, 1, -1, 291, 290]),   # empty, one, two inactive
    (Case(3, 16, 1, 700, 5, 650, 2, 8, 32, []), 12, 680, [128, 127, 129]),        # 192 columns; tile ends
    (Case(1, 8, 8, 2600, 30, 2500, 4, 4, 64, [0, 1]), 1, 2550, None),             # a single token
    (Case(40, 4, 4, 200, 16, 144, 4, 2, 64, [2]), 4, 150, None),                  # 160 (sequence, head) pairs
    (Case(1, 256, 2, 300, 3, 200, 8, 2, 64, []), 5, 210, None),                   # 640 columns per KV head
]


@pytest.mark.parametrize("ci", range(len(CASES)))
def test_tree_matches_reference(cuda_dev, kvq, ci):
    c, n_q, T, lens = CASES[ci]
    F = Filled(c, 3000 + 10 * ci, cuda_dev)
    q = bf16((c.B, n_q, c.H_q, c.D), 3003 + 10 * ci, cuda_dev)
    kd, vd = _drafts(c, n_q, 3004 + 10 * ci, cuda_dev)
    masks = random_tree(n_q, c.B, 7 + ci)
    out, lse = _call(F, q, kd, vd, masks, T, lens)
    check_tree(c, out, lse, f64(q), F.khat, F.vhat, f64(kd), f64(vd), masks, _active(lens or [T] * c.B, T))


def test_tree_faint_tail(cuda_dev, kvq):
    """One draft outweighs 63 others by e^17 each and holds zeros where they
    hold ones: the output is their share.  A weight is off by half a step of
    fp16's subnormals (2^-25) from P = 2^3 e^-17, and the output rounded once."""
    c = Case(1, 2, 1, 100, 4, 60, 4, 4, 64, [])
    F = Filled(c, 3900, cuda_dev)
    q = torch.zeros(1, 64, 2, 128, dtype=torch.bfloat16, device=cuda_dev)
    q[..., 0] = 1.0 / SCALE
    assert float(q[0, 0, 0, 0]) * SCALE == pytest.approx(1.0, abs=2.0 ** -8)
    gap = float(q[0, 0, 0, 0]) * SCALE * 17.0
    kd = torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device=cuda_dev)
    vd = torch.ones_like(kd)
    kd[:, :, 40, 0], vd[:, :, 40] = 17.0, 0.0
    out, lse = _call(F, q, kd, vd, np.full((1, 64), -1, np.int64).view(np.uint64), 0)
    w = np.exp(-gap)
    want = 63 * w / (1 + 63 * w)
    tol = 2.0 ** -25 / (2.0 ** 3 * w) + 2.0 ** -8 + 2.0 ** -16
    assert np.all(np.abs(f64(out) / want - 1.0) <= tol)
    assert np.all(np.abs(f64(lse) - gap - np.log1p(63 * w)) <= 2.0 ** -19 * gap)


BITS = [(kb, vb, G) for kb in (2, 4, 8, 16) for vb in (2, 4, 8, 16) for G in (32, 64, 128)]


@pytest.mark.parametrize("kb,vb,G", BITS)
def test_tree_every_width(cuda_dev, kvq, kb, vb, G):
    """Every pair of widths and group size, with the three kinds of heads,
    loud K channels, a text prefix and suffix."""
    c = Case(1, 9, 3, 330, 13, 300, kb, vb, G, [1], konly=[2])
    F = Filled(c, 3300, cuda_dev)
    k = F.k.clone()
    k[..., [3, 40, 77, 126]] *= 10
    kvq.quantize_append(F.L, F.cache, k, F.v, 0)
    import oracle
    khat = oracle.reconstruct(bits(k), c.vs, c.ve, c.mask(), kb, G)[0]
    q, (kd, vd) = bf16((1, 6, 9, 128), 3303, cuda_dev), _drafts(c, 6, 3304, cuda_dev)
    masks = random_tree(6, 1, 5)
    out, lse = _call(F, q, kd, vd, masks, 321)
    check_tree(c, out, lse, f64(q), khat, F.vhat, f64(kd), f64(vd), masks, [321])


def test_tree_masks(cuda_dev, kvq):
    """A chain, all drafts, no draft (the context alone), bits past n_q, and
    with an empty context rows that attend nothing."""
    c = Case(2, 6, 2, 300, 10, 250, 4, 4, 32, [0])
    F = Filled(c, 3400, cuda_dev)
    n_q = 5
    q, (kd, vd) = bf16((2, n_q, 6, 128), 3403, cuda_dev), _drafts(c, n_q, 3404, cuda_dev)
    chain = np.array([[(1 << (i + 1)) - 1 for i in range(n_q)]], np.uint64)
    for masks in (chain, np.full((1, n_q), 31, np.uint64), np.zeros((2, n_q), np.uint64),
                  np.array([[1, 2, 0, 0xFFFFFFFFFFFFFFE8, 0], [0, 0, 31, 16, 1]], np.uint64)):
        for lens in ([270, 270], [0, 0], [0, 13]):
            out, lse = _call(F, q, kd, vd, masks, 270, lens)
            low = masks & np.uint64(31)
            check_tree(c, out, lse, f64(q), F.khat, F.vhat, f64(kd), f64(vd), low, lens)
    out, lse = _call(F, q, kd, vd, np.zeros((1, n_q), np.uint64), 0)   # T_ctx = 0
    assert not out.float().abs().any() and torch.isneginf(lse).all()


def test_tree_ignores_what_no_token_attends(cuda_dev, kvq):
    """NaN and infinities in drafts that nobody attends, in cache rows past
    the context, and in the queries of other columns."""
    c = Case(2, 4, 2, 300, 10, 200, 8, 8, 64, [1])
    F = Filled(c, 3500, cuda_dev)
    n_q, T = 7, 233
    q, (kd, vd) = bf16((2, n_q, 4, 128), 3503, cuda_dev), _drafts(c, n_q, 3504, cuda_dev)
    masks = random_tree(n_q, 2, 3)
    keep = [0, 1, 2, 4]
    bad = [j for j in range(n_q) if j not in keep]
    for j in bad:
        masks &= np.uint64(~(1 << j) & 0xFFFFFFFFFFFFFFFF)
    want = (f64(q), f64(kd), f64(vd))
    nan = torch.tensor([float("nan"), float("inf"), -float("inf")], device=cuda_dev)
    for i, j in enumerate(bad):
        kd[:, :, j] = nan[i % 3]
        vd[:, :, j] = nan[(i + 1) % 3]
    late = torch.full((2, 2, 300 - T, 128), float("nan"), dtype=torch.bfloat16, device=cuda_dev)
    kvq.quantize_append(F.L, F.cache, late, late, T)
    out, lse = _call(F, q, kd, vd, masks, T)
    check_tree(c, out, lse, want[0], F.khat, F.vhat, want[1], want[2], masks, [T, T])
    q[:, 5] = float("nan")   # a padded token: only its own rows
    out, lse = _call(F, q, kd, vd, masks, T)
    ok = [i for i in range(n_q) if i != 5]
    check_tree(c, out[:, ok], lse[:, ok], want[0][:, ok], F.khat, F.vhat, want[1], want[2], masks[:, ok], [T, T])


def test_tree_strides_shared_mask_no_lse(cuda_dev, kvq):
    """Drafts inside larger tensors, one mask for the batch, no lse, and a
    second call on the same workspace: the same bits."""
    c = Case(3, 8, 4, 260, 10, 200, 4, 2, 64, [2])
    F = Filled(c, 3600, cuda_dev)
    n_q, T = 11, 222
    q = bf16((3, n_q, 8, 128), 3601, cuda_dev)
    wide = bf16((3, n_q + 2, 2, 5, 136), 3602, cuda_dev)[:, 1:-1, :, :4, 8:]
    kd, vd = wide[:, :, 0].transpose(1, 2), wide[:, :, 1].transpose(1, 2)
    masks = random_tree(n_q, 1, 8)
    ws = torch.zeros(kvq.decode_tree_workspace_bytes(F.L, n_q), dtype=torch.uint8, device=cuda_dev)
    out, _ = _call(F, q, kd, vd, masks, T, lse=False, ws=ws)
    check_tree(c, out, None, f64(q), F.khat, F.vhat, f64(kd), f64(vd), masks, [T] * 3)
    again, _ = _call(F, q, kd.contiguous(), vd.contiguous(), masks, T, [T] * 3, ws=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_tree_chain_is_multi_query_decode(cuda_dev, kvq):
    """A chain of drafts equals kvq_decode_attention_mq with the same rows
    appended, within both calls' roundings."""
    c = Case(2, 14, 2, 900, 14, 840, 4, 2, 64, [0])
    F = Filled(c, 3700, cuda_dev)
    n_q, T = 6, 860
    q = bf16((2, n_q, 14, 128), 3701, cuda_dev)
    kd, vd = F.k[:, :, T:T + n_q], F.v[:, :, T:T + n_q]
    masks = np.array([[(1 << (i + 1)) - 1 for i in range(n_q)]], np.uint64)
    out, lse = _call(F, q, kd, vd, masks, T)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.zeros(kvq.decode_mq_workspace_bytes(F.L, n_q), dtype=torch.uint8, device=cuda_dev)
    kvq.decode_attention_mq(F.L, F.cache, q, T + n_q, o2, SCALE, l2, ws)
    torch.cuda.synchronize()
    check_tree(c, out, lse, f64(q), F.khat, F.vhat, f64(kd), f64(vd), masks, [T, T])
    vmax = float(F.v.float().abs().max())
    assert float((out.float() - o2.float()).abs().max()) <= 2 * 2.0 ** -8 * vmax
    assert float((lse - l2).abs().max()) <= 1e-3


@pytest.mark.parametrize("n_q,T", [(16, 6300), (3, 6287), (40, 6293)])
def test_tree_llava_ov_layer(cuda_dev, kvq, n_q, T):
    """The LLaVA-OneVision-7B layer (28/4 heads, 14 text + 6273 visual
    positions, K4/V2 G64, head 0 in bf16)."""
    c = Case(1, 28, 4, 6400, 14, 14 + 6273, 4, 2, 64, [0])
    F = Filled(c, 3800, cuda_dev)
    q, (kd, vd) = bf16((1, n_q, 28, 128), 3803, cuda_dev), _drafts(c, n_q, 3804, cuda_dev)
    masks = random_tree(n_q, 1, 11)
    out, lse = _call(F, q, kd, vd, masks, T)
    check_tree(c, out, lse, f64(q), F.khat, F.vhat, f64(kd), f64(vd), masks, [T])


def test_tree_peaked_scores(cuda_dev, kvq):
    """Scores far apart, rising and falling along the cache (the running
    maximum moves by hundreds), and one position that takes all the weight."""
    c = Case(1, 4, 2, 1200, 10, 1100, 8, 8, 128, [])
    F = Filled(c, 3900, cuda_dev)
    n_q, T = 4, 1180
    ramp = torch.linspace(-40, 40, c.T_cap, device=cuda_dev)
    for sign in (1, -1):
        k = (F.k.float() * 0.1 + sign * ramp[:, None]).to(torch.bfloat16)
        kvq.quantize_append(F.L, F.cache, k, F.v, 0)
        import oracle
        khat = oracle.reconstruct(bits(k), c.vs, c.ve, c.mask(), c.kb, c.G)[0]
        q, (kd, vd) = bf16((1, n_q, 4, 128), 3903, cuda_dev), _drafts(c, n_q, 3904, cuda_dev)
        q = (q.float() * 0.2 + 1).to(torch.bfloat16)
        masks = random_tree(n_q, 1, 2)
        out, lse = _call(F, q, kd, vd, masks, T)
        check_tree(c, out, lse, f64(q), khat, F.vhat, f64(kd), f64(vd), masks, [T])


COMMITS = [
    # layout, n_q, T_ctx, lengths, path lengths
    (Case(1, 4, 1, 300, 14, 256, 4, 4, 32, []), 5, 257, None, [3]),
    (Case(4, 8, 4, 300, 10, 250, 8, 4, 32, [1], konly=[2]), 8, 290, [250, 290, 0, 2], [8, 8, 8, 8]),
    # inactive: into the visual block, past T_cap, length -1, length past T_ctx, path lengths -1 and 9, inside the visual block
    (Case(7, 8, 2, 300, 10, 250, 8, 4, 32, []), 8, 298, [5, 297, -1, 299, 260, 260, 100], [6, 4, 2, 2, -1, 9, 1]),
    (Case(2, 6, 2, 64, 0, 0, 2, 2, 32, []), 64, 20, [0, 0], [0, 64]),
]


@pytest.mark.parametrize("ci", range(len(COMMITS)))
def test_commit_stores_the_path(cuda_dev, kvq, ci):
    c, n_q, T, lens, counts = COMMITS[ci]
    F = Filled(c, 4000 + ci, cuda_dev)
    kd, vd = _drafts(c, n_q, 4010 + ci, cuda_dev)
    g = np.random.default_rng(ci)
    m = n_q
    path = g.integers(0, n_q, (c.B, m)).astype(np.int32)   # any order, repeats
    for b, n in enumerate(counts):
        path[b, max(0, min(n, m)):] = -7                       # unread
    want = F.cache.clone()
    at = lens or [T] * c.B
    new = []
    for b in range(c.B):
        n, t = counts[b], at[b]
        ok = 0 <= t <= T and 0 <= n <= m and t + n <= c.T_cap and not (n and c.vs < c.ve and t < c.ve and t + n > c.vs)
        new.append(t + n if ok else -1)
        for k in range(n if ok else 0):
            j = int(path[b, k])
            one = F.L.d
            row = t + k if t < c.ve else t + k - int(F.L.Tv)
            for seg, x in ((kvq.SEG_TEXT_K, kd), (kvq.SEG_TEXT_V, vd)):
                for h in range(c.H_kv):
                    o = int(F.L.off[seg]) + 256 * ((b * one.H_kv + h) * int(F.L.T_text) + row)
                    want[o:o + 256] = x[b, h, j].contiguous().view(torch.uint8)
    nl = torch.full((c.B,), 99, dtype=torch.int32, device=cuda_dev)
    kvq.tree_commit(F.L, F.cache, kd, vd, torch.from_numpy(path).to(cuda_dev),
                    torch.tensor(counts, dtype=torch.int32, device=cuda_dev), T,
                    None if lens is None else torch.tensor(lens, dtype=torch.int32, device=cuda_dev), nl)
    torch.cuda.synchronize()
    assert nl.tolist() == new
    assert torch.equal(F.cache, want)


def test_commit_refuses_a_bad_path_entry(cuda_dev, kvq):
    """An index outside the drafts makes its sequence inactive, the others not."""
    c = Case(3, 4, 2, 100, 4, 60, 4, 4, 64, [])
    F = Filled(c, 4100, cuda_dev)
    kd, vd = _drafts(c, 5, 4101, cuda_dev)
    path = torch.tensor([[0, 5], [1, 2], [-1, 0]], dtype=torch.int32, device=cuda_dev)
    n = torch.tensor([2, 2, 1], dtype=torch.int32, device=cuda_dev)
    nl = torch.zeros(3, dtype=torch.int32, device=cuda_dev)
    before = F.cache.clone()
    kvq.tree_commit(F.L, F.cache, kd, vd, path, n, 70, new_len=nl)
    torch.cuda.synchronize()
    assert nl.tolist() == [-1, 72, -1]
    rows = slice(int(F.L.off[kvq.SEG_TEXT_K]), int(F.L.off[kvq.SEG_TEXT_K]) + 3 * 2 * int(F.L.T_text) * 256)
    changed = (F.cache != before)[rows].view(3, 2, -1, 256).any(-1)
    assert not changed[0].any() and not changed[2].any()
    assert changed[1, :, 14:16].all() and int(changed.sum()) == 4
