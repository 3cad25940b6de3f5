"""kvq_decode_attention_window against attention in 64 bits over the positions
that each token sees."""
import numpy as np
import pytest
import torch

from gpu_helpers import Case
from serving_ref import Filled, bf16, f64
from step_ref import check_window

pytestmark = pytest.mark.gpu


def run(kvq, dev, f, q, T, n_sink, window, lens=None, scale=None, lse=True):
    out = torch.full_like(q, 7.0)
    l = torch.full(q.shape[:3], 7.0, device=dev) if lse else None
    kvq.decode_attention_window(f.L, f.cache, q, T, n_sink, window, out, scale, l,
                                None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev))
    return out, l


# B, H_q, H_kv, T_cap, vs, ve, kb, vb, G, prot
LAYOUTS = [
    Case(2, 8, 2, 300, 14, 256, 4, 2, 64, [0]),
    Case(1, 12, 4, 200, 5, 170, 8, 4, 32, [2], konly=[0]),
    Case(3, 3, 3, 150, 0, 100, 2, 2, 128, []),
    Case(1, 7, 1, 260, 33, 240, 16, 2, 32, []),
    Case(2, 4, 4, 130, 20, 20, 4, 4, 32, [1]),      # text alone
    Case(1, 10, 2, 140, 0, 140, 4, 16, 64, [1]),    # visual to the end
]


@pytest.mark.parametrize("n_q", [1, 3, 17])
@pytest.mark.parametrize("ci", range(len(LAYOUTS)))
def test_window_matches_reference(cuda_dev, kvq, ci, n_q):
    c = LAYOUTS[ci]
    f = Filled(c, 60 + ci, cuda_dev)
    q = bf16((c.B, n_q, c.H_q, 128), 70 + ci, cuda_dev)
    T = c.T_cap - 3
    for n_sink, window in ((0, 1), (4, 50), (37, 16), (0, T), (T, 1), (60, T - 61), (1, 2 ** 31 - 1), (2 ** 31 - 1, 5)):
        out, lse = run(kvq, cuda_dev, f, q, T, n_sink, window)
        check_window(c, out, lse, f64(q), f.khat, f.vhat, [T] * c.B, n_sink, window)


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("vb", [2, 4, 8, 16])
@pytest.mark.parametrize("kb", [2, 4, 8, 16])
def test_window_every_width(cuda_dev, kvq, kb, vb, G):
    c = Case(2, 6, 3, 230, 9, 210, kb, vb, G, [1], konly=[2])
    f = Filled(c, 3, cuda_dev)
    for n_q in (1, 6):  # one and two tiles of columns
        q = bf16((c.B, n_q, c.H_q, 128), 4, cuda_dev)
        out, lse = run(kvq, cuda_dev, f, q, 225, 21, 130, lens=[225, 214])
        check_window(c, out, lse, f64(q), f.khat, f.vhat, [225, 214], 21, 130)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100])
def test_window_short_sequences(cuda_dev, kvq, T):
    """Every length around a block, the first positions and the window apart,
    next to one another and overlapping; tokens before the first position see nothing."""
    c = Case(1, 5, 1, 100, 10, 60, 4, 4, 32, [])
    f = Filled(c, 5, cuda_dev)
    for n_q in (1, 2, 5):
        q = bf16((1, n_q, 5, 128), 6, cuda_dev)
        for n_sink, window in ((0, 3), (7, 9), (30, 30), (1, 100)):
            out, lse = run(kvq, cuda_dev, f, q, T, n_sink, window)
            check_window(c, out, lse, f64(q), f.khat, f.vhat, [T], n_sink, window)


def test_window_lengths_per_sequence(cuda_dev, kvq):
    """Lengths on the device: inactive entries, 0, lengths inside the visual block."""
    c = Case(8, 8, 2, 300, 30, 260, 4, 2, 64, [1])
    f = Filled(c, 7, cuda_dev)
    q = bf16((8, 4, 8, 128), 8, cuda_dev)
    lens = [290, 0, -1, 291, 1, 31, 200, 263]
    out, lse = run(kvq, cuda_dev, f, q, 290, 16, 64, lens=lens)
    check_window(c, out, lse, f64(q), f.khat, f.vhat, [None if n < 0 or n > 290 else n for n in lens], 16, 64)
    for b in (1, 2, 3):
        assert (out[b] == 0).all() and torch.isneginf(lse[b]).all()
    # no lse wanted: the same rows
    assert torch.equal(run(kvq, cuda_dev, f, q, 290, 16, 64, lens=lens, lse=False)[0], out)


def test_window_ignores_what_no_token_attends(cuda_dev, kvq):
    """Rows between the first positions and the window, and behind the end, may hold anything."""
    c = Case(1, 8, 2, 400, 20, 350, 8, 2, 32, [1])
    f = Filled(c, 9, cuda_dev)
    q = bf16((1, 3, 8, 128), 10, cuda_dev)
    T, n_sink, window = 380, 25, 100
    out, lse = run(kvq, cuda_dev, f, q, T, n_sink, window)
    # NaN in all unseen rows: an image of the cache is built from rows that are NaN there
    lo = T - 3 - window + 1
    L, img = f.L, f.cache.clone()
    for key, (codes, sz, plain, text) in ((True, (0, 1, 4, 6)), (False, (2, 3, 5, 7))):
        for s in (codes, sz, plain, text):
            rows, w = (int(L.Tv_pad) if s < 4 else (int(L.Tv) if s < 6 else int(L.T_text))), int(L.row_bytes[s])
            if not w or not int(L.bytes[s]):
                continue
            v = img[int(L.off[s]):int(L.off[s]) + int(L.bytes[s])].view(-1, rows, w)
            if s < 6:
                v[:, n_sink - c.vs:lo - c.vs] = 0xFF
                v[:, c.ve - c.vs:] = 0xFF
            else:
                v[:, T - int(L.Tv):] = 0xFF
    f.cache.copy_(img)
    again = run(kvq, cuda_dev, f, q, T, n_sink, window)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_window_is_full_attention(cuda_dev, kvq):
    """A window over everything is kvq_decode_attention_mq up to roundings."""
    c = Case(2, 28, 4, 1500, 14, 1400, 4, 2, 64, [0])
    f = Filled(c, 11, cuda_dev)
    q = bf16((2, 4, 28, 128), 12, cuda_dev)
    out, lse = run(kvq, cuda_dev, f, q, 1450, 0, 1450)
    ref, rl = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.zeros(kvq.decode_mq_workspace_bytes(f.L, 4), dtype=torch.uint8, device=cuda_dev)
    kvq.decode_attention_mq(f.L, f.cache, q, 1450, ref, None, rl, ws)
    assert (out.float() - ref.float()).abs().max() < 8e-3 * np.abs(f.vhat).max() and (lse - rl).abs().max() < 2e-3
    check_window(c, out, lse, f64(q), f.khat, f.vhat, [1450] * 2, 0, 1450)


@pytest.mark.parametrize("n_q,T,window", [(1, 6300, 2048), (16, 6300, 1000), (1, 6290, 6000), (64, 6350, 300)])
def test_window_llava_ov_layer(cuda_dev, kvq, n_q, T, window):
    c = Case(1, 28, 4, 6400, 14, 6287, 4, 2, 64, [0])
    f = Filled(c, 13, cuda_dev)
    q = bf16((1, n_q, 28, 128), 14, cuda_dev)
    out, lse = run(kvq, cuda_dev, f, q, T, 30, window)
    check_window(c, out, lse, f64(q), f.khat, f.vhat, [T], 30, window)


@pytest.mark.parametrize("vb,G", [(2, 32), (8, 128)])
def test_window_faint_weights_beside_a_sink(cuda_dev, kvq, vb, G):
    """One first position takes most of the mass; thousands of window positions
    of weight 2^-14 of it each carry the rest, all of one sign."""
    c = Case(1, 2, 1, 9000, 4, 8990, 16, vb, G, [])
    from gpu_helpers import alloc_cache, append, bits
    import oracle
    f = Filled.__new__(Filled)
    f.c, f.L = c, c.layout()
    f.k = torch.zeros(1, 1, 9000, 128, dtype=torch.bfloat16, device=cuda_dev)
    f.k[:, :, 0, 0] = 8.0
    f.v = bf16((1, 1, 9000, 128), 15, cuda_dev, 0.25).abs() + 1
    f.v[:, :, 0] = -3.0
    f.v = f.v.bfloat16()
    f.cache = alloc_cache(f.L, cuda_dev)
    append(f.L, f.cache, f.k, f.v, 0)
    f.khat = oracle.reconstruct(bits(f.k), c.vs, c.ve, c.mask(), c.kb, c.G)[0]
    f.vhat = oracle.reconstruct(bits(f.v), c.vs, c.ve, [0], c.vb, c.G)[0]
    q = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16, device=cuda_dev)
    q[..., 0] = 14.0  # 8 * 14 / sqrt(128) = 9.9: e^9.9 = 2^14.3
    out, lse = run(kvq, cuda_dev, f, q, 8995, 1, 8192)
    check_window(c, out, lse, f64(q), f.khat, f.vhat, [8995], 1, 8192)


@pytest.mark.parametrize("vs", [1e-30, 2.0 ** -20, 300.0, 60000.0])
@pytest.mark.parametrize("vb", [2, 8, 16])
def test_window_values_of_any_size(cuda_dev, kvq, vb, vs):
    """V from tiny (bf16 rows alone: packed scales are fp16) to the largest."""
    c = Case(1, 4, 2, 300, 10, 250, 4, vb, 32, [1])
    f = Filled(c, 16, cuda_dev)
    unit = f.v.float() / f.v.float().abs().max()
    v = (unit * vs).bfloat16()
    if vs < 2.0 ** -14:
        v = torch.where(torch.arange(300, device=cuda_dev)[None, None, :, None].expand_as(v) < 250, torch.zeros_like(v), v)
    import oracle
    from gpu_helpers import append, bits
    append(f.L, f.cache, f.k, v, 0)
    vhat = oracle.reconstruct(bits(v), c.vs, c.ve, [0, 1], c.vb, c.G)[0]
    q = bf16((1, 2, 4, 128), 17, cuda_dev)
    out, lse = run(kvq, cuda_dev, f, q, 299, 12, 270)
    check_window(c, out, lse, f64(q), f.khat, vhat, [299], 12, 270, codes=vs > 1 and vb < 16)


@pytest.mark.parametrize("qs,scale", [(1e-20, 1e20), (2.0 ** 40, 2.0 ** -40), (1.0, 0.0), (1.0, -0.3), (30.0, 0.5)])
def test_window_scores_of_any_size(cuda_dev, kvq, qs, scale):
    c = Case(1, 8, 2, 200, 10, 150, 4, 4, 32, [1])
    f = Filled(c, 18, cuda_dev)
    q = (bf16((1, 2, 8, 128), 19, cuda_dev).float() * qs).bfloat16()
    out, lse = run(kvq, cuda_dev, f, q, 180, 8, 100, scale=scale)
    check_window(c, out, lse, f64(q), f.khat, f.vhat, [180], 8, 100, scale)


def test_window_query_that_is_not_finite(cuda_dev, kvq):
    """A NaN in a query makes its own row NaN and no other."""
    c = Case(2, 8, 2, 200, 10, 150, 2, 4, 32, [1])
    f = Filled(c, 20, cuda_dev)
    q = bf16((2, 3, 8, 128), 21, cuda_dev)
    good = run(kvq, cuda_dev, f, q, 180, 8, 100)
    q[1, 1, 2, 5] = float("nan")
    out, lse = run(kvq, cuda_dev, f, q, 180, 8, 100)
    assert torch.isnan(out[1, 1, 2]).all() and torch.isnan(lse[1, 1, 2])
    out[1, 1, 2], lse[1, 1, 2] = good[0][1, 1, 2], good[1][1, 1, 2]
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])


def test_window_many_units(cuda_dev, kvq):
    """More units than one wave of clusters, and one CTA a unit."""
    c = Case(40, 32, 16, 180, 8, 160, 4, 4, 64, [3])
    f = Filled(c, 22, cuda_dev)
    q = bf16((40, 2, 32, 128), 23, cuda_dev)
    out, lse = run(kvq, cuda_dev, f, q, 175, 6, 90)
    check_window(c, out, lse, f64(q), f.khat, f.vhat, [175] * 40, 6, 90)


def test_window_is_repeatable(cuda_dev, kvq):
    c = Case(2, 28, 4, 3000, 14, 2900, 2, 2, 32, [0])
    f = Filled(c, 24, cuda_dev)
    q = bf16((2, 2, 28, 128), 25, cuda_dev)
    a, b = run(kvq, cuda_dev, f, q, 2950, 10, 1024), run(kvq, cuda_dev, f, q, 2950, 10, 1024)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("prot", [[], list(range(8))])
def test_window_cache_past_32_bits(cuda_dev, kvq, prot):
    """A cache of 4.9 GB, rows of the last head more than 2^32 bytes in (bf16
    rows, so that the reference reads them from the buffer)."""
    T = 1200000
    c = Case(1, 16, 8, T, 3, T - 7, 16, 16, 32, prot)
    L = c.layout()
    assert int(L.total_bytes) > 2 ** 32 + 2 ** 28
    cache = torch.empty(int(L.total_bytes), dtype=torch.uint8, device=cuda_dev)
    g = torch.Generator(device=cuda_dev).manual_seed(5)
    cache.view(torch.bfloat16).normal_(generator=g)

    def rows(vis, text):
        """[8, T, 128] of the last 8,000 positions and the first 16, fp64."""
        s = vis[1] if prot else vis[0]
        n = int(L.Tv) if prot else int(L.Tv_pad)
        v = cache[int(L.off[s]):int(L.off[s]) + 8 * n * 256].view(torch.bfloat16).view(8, n, 128)
        t = cache[int(L.off[text]):int(L.off[text]) + 8 * int(L.T_text) * 256].view(torch.bfloat16).view(8, int(L.T_text), 128)
        first = torch.cat([t[:, :3], v[:, :13]], 1)
        last = torch.cat([v[:, T - 8000 - 3:T - 10], t[:, 3:]], 1)
        return f64(first), f64(last)

    q = bf16((1, 2, 16, 128), 40, cuda_dev)
    out, lse = torch.zeros_like(q), torch.zeros(1, 2, 16, device=cuda_dev)
    kvq.decode_attention_window(L, cache, q, T, 16, 7000, out, None, lse)
    (k0, k1), (v0, v1) = rows((kvq.SEG_K_CODES, kvq.SEG_PROT_K), kvq.SEG_TEXT_K), rows((kvq.SEG_V_CODES, kvq.SEG_PROT_V), kvq.SEG_TEXT_V)
    # the same positions as a short sequence: the first 16, then the last 8,000
    small = Case(1, 16, 8, 8016, 3, 8009, 16, 16, 32, prot)
    check_window(small, out, lse, f64(q), np.concatenate([k0, k1], 1)[None], np.concatenate([v0, v1], 1)[None], [8016], 16, 7000)


def test_window_of_a_long_context(cuda_dev, kvq):
    """150,000 positions in the window of one 2-bit head: several turns of every ring."""
    c = Case(1, 3, 1, 160000, 5, 159000, 2, 2, 128, [])
    f = Filled(c, 41, cuda_dev)
    q = bf16((1, 2, 3, 128), 42, cuda_dev)
    out, lse = run(kvq, cuda_dev, f, q, 159500, 33, 150000)
    check_window(c, out, lse, f64(q), f.khat, f.vhat, [159500], 33, 150000)
