"""kvq_norm_rope against its formula in 64 bits: axes, partial rotations, both
pairings, strides, in place, odd and single tokens, far positions."""
import numpy as np
import pytest
import torch

import synth
from serving_ref import bf16, f64
from step_ref import check_rope

pytestmark = pytest.mark.gpu


def _freq(rot, base=1e6):
    return (base ** (-np.arange(rot // 2) * 2.0 / rot)).astype(np.float32)


def _layout(kvq, B, Hq, Hkv):
    return kvq.cache_layout(B, Hq, Hkv, 128, 16, 0, 0, 4, 4, 32)


def _pos(n_axes, B, n, far, seed):
    return np.random.default_rng(seed).integers(0, far, (n_axes, B, n)).astype(np.int32)


def _run(kvq, dev, B, n, Hq, Hkv, rot, axis, pair, norm, far, seed, eps=1e-6):
    q, k = bf16((B, n, Hq, 128), seed, dev), bf16((B, n, Hkv, 128), seed + 1, dev)
    wq, wk = (1 + 0.5 * bf16((128,), seed + 2, dev), 1 + 0.5 * bf16((128,), seed + 3, dev)) if norm else (None, None)
    pos, freq = _pos(max(axis) + 1, B, n, far, seed), _freq(rot)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    kvq.norm_rope(_layout(kvq, B, Hq, Hkv), kvq.rope_desc(rot, axis, pair), q, k, torch.from_numpy(pos).to(dev),
                  torch.from_numpy(freq).to(dev), qo, ko, wq, wk, eps)
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        check_rope(got, f64(x), pos, freq.astype(np.float64), axis, rot, pair, None if w is None else f64(w), eps)


SECTIONS = [0] * 16 + [1] * 24 + [2] * 24
CASES = [
    # B, n, Hq, Hkv, rot, axis, interleaved, norm, positions below
    (1, 1, 28, 4, 128, SECTIONS, False, False, 6300),
    (1, 1, 1, 1, 128, [0] * 64, True, True, 2),
    (2, 7, 5, 5, 128, SECTIONS, False, True, 40000),
    (3, 33, 6, 2, 96, [0] * 48, True, True, 33000),
    (2, 19, 4, 4, 8, [0, 1, 2, 3], False, False, 1000),
    (1, 5, 3, 3, 8, [3, 0, 0, 1], True, True, 1000),
    (2, 101, 40, 8, 64, [1] * 20 + [0] * 12, False, True, 200000),
    (1, 640, 28, 4, 128, SECTIONS, False, True, 6300),       # groups of four and eight heads
    (4, 300, 32, 32, 120, [i % 3 for i in range(60)], True, False, 2 ** 31 - 1),
    (2, 9, 128, 128, 40, [0] * 20, False, True, 5),
]


@pytest.mark.parametrize("ci", range(len(CASES)))
def test_rope_matches_formula(cuda_dev, kvq, ci):
    B, n, Hq, Hkv, rot, axis, pair, norm, far = CASES[ci]
    _run(kvq, cuda_dev, B, n, Hq, Hkv, rot, axis, pair, norm, far, 40 + ci)


def test_rope_strides_in_place_and_one_side(cuda_dev, kvq):
    """The heads as parts of one projection's output, written where they are or
    into the cache calls' order; one side alone leaves the rest as it was."""
    B, n, Hq, Hkv, rot = 2, 37, 6, 3, 128
    qkv = bf16((B, n, Hq + 2 * Hkv, 128), 5, cuda_dev)
    start, L, R = qkv.clone(), _layout(kvq, B, Hq, Hkv), kvq.rope_desc(rot, SECTIONS)
    pos, freq = _pos(3, B, n, 9000, 6), _freq(rot)
    p, f = torch.from_numpy(pos).to(cuda_dev), torch.from_numpy(freq).to(cuda_dev)
    qv, kv = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
    ko = torch.zeros(B, Hkv, n, 128, dtype=torch.bfloat16, device=cuda_dev)
    kvq.norm_rope(L, R, None, kv, p, f, None, ko.transpose(1, 2))
    assert torch.equal(qkv, start)
    kvq.norm_rope(L, R, qv, kv, p, f, qv, kv)
    assert torch.equal(qkv[:, :, Hq + Hkv:], start[:, :, Hq + Hkv:])
    assert torch.equal(kv, ko.transpose(1, 2))
    for got, at in ((qv, slice(0, Hq)), (kv, slice(Hq, Hq + Hkv))):
        check_rope(got, f64(start[:, :, at]), pos, freq.astype(np.float64), SECTIONS, rot, False, None, 0.0)
    # one row of positions for the whole batch, and a slice of a longer one
    alone = torch.empty_like(start[:, :, :Hq])
    kvq.norm_rope(L, R, start[:, :, :Hq], None, p[:, 0], f, alone, None)
    check_rope(alone, f64(start[:, :, :Hq]), np.repeat(pos[:, :1], B, 1), freq.astype(np.float64), SECTIONS, rot, False, None, 0.0)
    long = torch.from_numpy(_pos(4, B, 2 * n, 9000, 7)).to(cuda_dev)
    kvq.norm_rope(L, R, start[:, :, :Hq], None, long[:, :, 5:5 + n], f, alone, None)
    check_rope(alone, f64(start[:, :, :Hq]), long[:, :, 5:5 + n].cpu().numpy(), freq.astype(np.float64), SECTIONS, rot, False, None, 0.0)


def test_rope_negative_positions_and_any_frequency(cuda_dev, kvq):
    """Positions below zero turn the other way; frequencies above a turn, below
    zero and zero are taken as they are."""
    B, n, H, rot = 1, 12, 2, 16
    x = bf16((B, n, H, 128), 8, cuda_dev)
    pos = np.array([0, 1, -1, 5, -7, 1000, -1000, 123456789, -123456789, 2 ** 31 - 1, -2 ** 31, 3], np.int32).reshape(1, 1, n)
    freq = np.array([1.0, -0.25, 0.0, 7.0, 1e-7, -20.5, 3.140625, 1e-3], np.float32)
    out = torch.empty_like(x)
    kvq.norm_rope(_layout(kvq, B, H, H), kvq.rope_desc(rot, [0] * 8), x, None, torch.from_numpy(pos).to(cuda_dev),
                  torch.from_numpy(freq).to(cuda_dev), out, None)
    # the reference's own angle is taken modulo a turn in long double (64-bit mantissa or better)
    turn = (pos[0, 0].astype(np.longdouble)[:, None] * freq.astype(np.longdouble)) % (2 * np.longdouble("3.14159265358979323846264338327950288"))
    y = f64(x)
    c, s = np.cos(turn.astype(np.float64))[None, :, None], np.sin(turn.astype(np.float64))[None, :, None]
    ref = y.copy()
    ref[..., :8], ref[..., 8:16] = y[..., :8] * c - y[..., 8:16] * s, y[..., 8:16] * c + y[..., :8] * s
    size = np.abs(y)
    size[..., :8] = size[..., 8:16] = np.abs(y[..., :8]) + np.abs(y[..., 8:16])
    # the turn is off by 2^31 * 2^-53 of itself at most: 20.5 * 2^-22 radians
    tol = 2.0 ** -7.99 * np.abs(ref) + (2.0 ** -18 + 20.5 * 2.0 ** -22) * size
    assert np.all(np.abs(f64(out) - ref) <= tol)


def test_rope_rows_of_any_size(cuda_dev, kvq):
    """Zero rows, tiny and huge ones; a NaN or an infinity stays in its row."""
    B, n, H = 1, 6, 2
    x = bf16((B, n, H, 128), 9, cuda_dev)
    x[0, 0] = 0
    x[0, 1] *= 2.0 ** -60
    x[0, 2] *= 2.0 ** 60
    x[0, 3, 0, 77] = float("nan")
    x[0, 4, 1, 3] = float("inf")
    w = torch.ones(128, dtype=torch.bfloat16, device=cuda_dev)
    pos, freq = _pos(1, B, n, 100, 1), _freq(128)
    out = torch.empty_like(x)
    for weight in (None, w):
        kvq.norm_rope(_layout(kvq, B, H, H), kvq.rope_desc(128, [0] * 64), x, None, torch.from_numpy(pos).to(cuda_dev),
                      torch.from_numpy(freq).to(cuda_dev), out, None, weight, None, 1e-6)
        fine = [(0, 0), (0, 1), (1, 0), (1, 1), (3, 1), (4, 0), (5, 0), (5, 1)] + ([(2, 0), (2, 1)] if weight is None else [])
        for t, h in fine:  # squares of 2^60 and more leave fp32
            check_rope(out[:, t:t + 1, h:h + 1], f64(x[:, t:t + 1, h:h + 1]), pos[:, :, t:t + 1], freq.astype(np.float64), [0] * 64,
                       128, False, None if weight is None else f64(weight), 1e-6)
        assert torch.isnan(out[0, 3, 0]).any()


def test_rope_feeds_a_decode_step(cuda_dev, kvq):
    """n = 1: the rows go straight into kvq_decode_step and come back from the cache."""
    from gpu_helpers import Case, alloc_cache
    c = Case(2, 8, 2, 64, 4, 40, 4, 4, 32, [1])
    L = c.layout()
    cache = alloc_cache(L, cuda_dev, 0)
    kvq.quantize_append(L, cache, bf16((2, 2, 50, 128), 1, cuda_dev), bf16((2, 2, 50, 128), 2, cuda_dev), 0)
    qkv = bf16((2, 1, 12, 128), 3, cuda_dev)
    q, k = torch.empty(2, 1, 8, 128, dtype=torch.bfloat16, device=cuda_dev), torch.empty(2, 1, 2, 128, dtype=torch.bfloat16, device=cuda_dev)
    pos = torch.full((3, 2, 1), 50, dtype=torch.int32, device=cuda_dev)
    kvq.norm_rope(L, kvq.rope_desc(128, SECTIONS), qkv[:, :, :8], qkv[:, :, 8:10], pos, torch.from_numpy(_freq(128)).to(cuda_dev), q, k)
    out, ws = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=cuda_dev), torch.zeros(int(L.workspace_bytes), dtype=torch.uint8, device=cuda_dev)
    kvq.decode_step(L, cache, q, k, qkv[:, 0, 10:].contiguous(), 50, out, None, None, ws)
    torch.cuda.synchronize()
    row = cache[int(L.off[kvq.SEG_TEXT_K]):][:int(L.bytes[kvq.SEG_TEXT_K])].view(torch.bfloat16).view(2, 2, -1, 128)[:, :, 50 - 36]
    assert torch.equal(row, k[:, 0]) and torch.isfinite(out).all()


def test_rope_rows_past_32_bits(cuda_dev, kvq):
    """Sequences and tokens more than 2^32 bytes apart, in and out."""
    B, n, H, rot = 2, 2, 3, 128
    x = bf16((B, n, H, 128), 30, cuda_dev)
    big = torch.empty(2 ** 31 + 2 ** 21, dtype=torch.bfloat16, device=cuda_dev)
    pos, freq = _pos(3, B, n, 9000, 31), _freq(rot)
    p, f = torch.from_numpy(pos).to(cuda_dev), torch.from_numpy(freq).to(cuda_dev)
    L, R = _layout(kvq, B, H, H), kvq.rope_desc(rot, SECTIONS)
    want = torch.empty_like(x)
    kvq.norm_rope(L, R, x, None, p, f, want, None)
    check_rope(want, f64(x), pos, freq.astype(np.float64), SECTIONS, rot, False, None, 0.0)
    for strides in ((2 ** 31 + 1024, 2 ** 19, 128, 1), (2 ** 19, 2 ** 31 + 4096, 2 ** 10, 1)):
        far = big.as_strided((B, n, H, 128), strides)
        far.copy_(x)
        out = torch.empty_like(x)
        kvq.norm_rope(L, R, far, None, p, f, out, None)
        assert torch.equal(out, want)
        kvq.norm_rope(L, R, far, None, p, f, far, None)
        assert torch.equal(far, want)
