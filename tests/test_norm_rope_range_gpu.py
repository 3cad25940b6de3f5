"""kvq_norm_rope at the ends of its range: normed rows whose squares leave fp32,
any eps, and frequencies of 2 and more at far positions."""
import numpy as np
import pytest
import torch

from serving_ref import bf16, f64
from step_ref import check_rope

pytestmark = pytest.mark.gpu
FREQ = (1e6 ** (-np.arange(64) / 64.0)).astype(np.float32)


def _layout(kvq, B, H):
    return kvq.cache_layout(B, H, H, 128, 16, 0, 0, 4, 4, 32)


@pytest.mark.parametrize("heads", [1, 3, 40])  # (with the tokens: one, four and eight heads a group)
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 1e30, 3e38])
def test_normed_rows_of_any_size(cuda_dev, kvq, eps, pair, heads):
    """y = x / sqrt(mean x^2 + eps) * w for rows from bf16's subnormals to its
    largest, huge and tiny ones in one launch, one element that takes the norm."""
    sizes = [2.0 ** e for e in (0, 62, 64, 70, 100, 126, -40, -62, -70, -76, -80, -100, -120, -126)]
    n = 2 * len(sizes) + 4
    n = n * (60 if heads == 40 else 1)
    x = bf16((1, n, heads, 128), 50, cuda_dev).float().clamp(-1.9, 1.9)
    for i, s in enumerate(sizes):
        x[0, i] *= s
        x[0, len(sizes) + i] *= 2.0 ** -30
        x[0, len(sizes) + i, :, 77] = s
    at = 2 * len(sizes)
    x[0, at] = 2.0 ** 128 - 2.0 ** 120           # every element the largest
    x[0, at + 1] = 2.0 ** -133 * torch.randint(1, 9, x[0, at + 1].shape, device=cuda_dev).float()  # subnormals
    x[0, at + 2, :, ::2] = -(2.0 ** 127)
    x = x.bfloat16()
    w = 1 + 0.25 * bf16((128,), 51, cuda_dev)
    pos = np.random.default_rng(52).integers(0, 9000, (1, 1, n)).astype(np.int32)
    out = torch.full_like(x, 7.0)
    kvq.norm_rope(_layout(kvq, 1, heads), kvq.rope_desc(128, [0] * 64, pair), x, None, torch.from_numpy(pos).to(cuda_dev),
                  torch.from_numpy(FREQ).to(cuda_dev), out, None, w, None, eps)
    check_rope(out, f64(x), pos, FREQ.astype(np.float64), [0] * 64, 128, pair, f64(w), float(np.float32(eps)))


def test_zero_rows_and_rows_that_are_not_finite(cuda_dev, kvq):
    """A zero row stays zero where eps is above 0; NaN and infinities stay in their rows."""
    x = bf16((1, 6, 2, 128), 53, cuda_dev)
    x[0, 0] = 0
    x[0, 1, 0, 5], x[0, 2, 1, 9] = float("nan"), float("inf")
    x[0, 3] *= 2.0 ** 100
    pos, w = torch.zeros(1, 1, 6, dtype=torch.int32, device=cuda_dev), torch.ones(128, dtype=torch.bfloat16, device=cuda_dev)
    L, R = _layout(kvq, 1, 2), kvq.rope_desc(128, [0] * 64)
    for eps in (1e-6, 1e-38):
        out = torch.empty_like(x)
        kvq.norm_rope(L, R, x, None, pos, torch.from_numpy(FREQ).to(cuda_dev), out, None, w, None, eps)
        assert (out[0, 0] == 0).all() and torch.isnan(out[0, 1, 0]).all() and torch.isnan(out[0, 2, 1, 9])
        for t, h in ((1, 1), (2, 0), (3, 0), (3, 1), (4, 0), (5, 1)):
            check_rope(out[:, t:t + 1, h:h + 1], f64(x[:, t:t + 1, h:h + 1]), np.zeros((1, 1, 1), np.int32), FREQ.astype(np.float64), [0] * 64, 128, False,
                       f64(w), eps)


def pi_bits(n):
    """floor(pi 2^n), by Machin's formula in integers."""
    def arctan(x):
        term = total = (1 << (n + 32)) // x
        k = 1
        while term:
            term //= -x * x
            k += 2
            total += term // k
        return total
    return (16 * arctan(5) - 4 * arctan(239)) >> 32


def turn(pos, f):
    """pos * f modulo 2 pi for an int and an fp32, exact to 2^-60 of a turn."""
    num, den = float(f).as_integer_ratio()
    two_pi = 2 * pi_bits(320)                                  # in units of 2^-320
    rest = ((int(pos) * num << 320) // den) % two_pi           # |pos f| < 2^159: off by 2^159 * 2^-318 of a turn
    return float(rest * (1 << 64) // two_pi) * 2.0 ** -64 * 2 * np.pi


@pytest.mark.parametrize("pair", [False, True])
def test_far_angles_of_any_frequency(cuda_dev, kvq, pair):
    """Angles are taken modulo a turn exactly: 2^-25 of a turn, whatever the
    position and the frequency (6.3 * 2^-25 < 2^-22), sine and cosine to 2^-21,
    two products and a sum: below 2^-19 of the pair, and one bf16 rounding."""
    freq = np.array([1.0, 1.9999999, 2.0, 3.1415927, 7.0, -20.5, 1000.0, 12345.678, -1e6, 16777215.0, 2.0 ** 31, 1e12, 2.0 ** 64, -1.2345e25,
                     2.0 ** 100 * 1.7, 3.4028235e38], np.float32)
    pos = np.array([0, 1, -1, 3, 1000, -999983, 123456789, 2 ** 30 + 1, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1, 2 ** 31 - 19], np.int32)
    n, rot = len(pos), 2 * len(freq)
    x = bf16((1, n, 2, 128), 54, cuda_dev)
    out = torch.empty_like(x)
    kvq.norm_rope(_layout(kvq, 1, 2), kvq.rope_desc(rot, [0] * len(freq), pair), x, None, torch.from_numpy(pos).to(cuda_dev).view(1, 1, n),
                  torch.from_numpy(freq).to(cuda_dev), out, None)
    a = np.array([[turn(p, f) for f in freq] for p in pos])[None, :, None]
    y = f64(x)
    i = np.arange(len(freq))
    p, q = (2 * i, 2 * i + 1) if pair else (i, i + len(freq))
    ref, size = y.copy(), np.abs(y)
    ref[..., p], ref[..., q] = y[..., p] * np.cos(a) - y[..., q] * np.sin(a), y[..., q] * np.cos(a) + y[..., p] * np.sin(a)
    size[..., p] = size[..., q] = np.abs(y[..., p]) + np.abs(y[..., q])
    err, tol = np.abs(f64(out) - ref), 2.0 ** -7.99 * np.abs(ref) + 2.0 ** -19 * size
    assert np.all(err <= tol), f"worst err / tol {np.max(err / tol):.3g}"
