"""Plain 64-bit references of the INT8 rows and products.

Every step that the header defines as rounded to 32 bits is formed in 64 bits
and rounded once, so codes, scales and the FP32 and bf16 products are compared
bit for bit; only SiLU*mul, whose exponential is the hardware's, has a
tolerance."""
import numpy as np

from nvfp4_w4a4_moe_quant_amd import datagen as D

F32, F64 = np.float32, np.float64


def quantize(x):
    """x float32 [rows, K] -> (codes int8, scales float32 [rows])."""
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(1)
        bad = ~np.isfinite(x).all(1)
        s = np.maximum((amax.astype(F64) / 127.0).astype(F32), F32(2.0 ** -126))
        s[amax == 0] = 0
        r = np.where(s > 0, 1.0 / s.astype(F64), 0.0).astype(F32)
        r[bad] = 0
        v = np.where(bad[:, None], 0, x) * r[:, None]     # one rounding to 32 bits
        s[bad] = np.nan
    assert v.dtype == F32 and (np.abs(np.rint(v)) <= 127).all()
    return np.rint(v).astype(np.int8), s


def product(a, sa, w, sw, offsets, gather=None):
    """y float32 [rows, N].  Sums of 8-bit products are exact in 64-bit floats."""
    rows, N = int(offsets[-1]), w.shape[1]
    y = np.zeros((rows, N), F32)
    for g in range(len(offsets) - 1):
        j = np.arange(offsets[g], offsets[g + 1])
        src = j if gather is None else gather[j]
        acc = a[src].astype(F64) @ w[g].astype(F64).T
        assert np.abs(acc).max(initial=0) < 2 ** 31
        with np.errstate(invalid="ignore", over="ignore"):
            y[j] = (sa[src][:, None] * sw[g][None, :]) * acc.astype(F32)
    return y


def bf16(y):
    """Nearest bf16, as float32."""
    return D.bf16_to_f32(D.bf16_bits(np.ascontiguousarray(y, F32)))


def silu_mul(y):
    """(h, tolerance) of the FP32 gate and up columns.  e^-g in hardware: the
    exponent's product with log2 e is off by |g| 2^-23 and the result by two
    steps of 2^-23, the sum, its reciprocal and the two products by less than
    six of 2^-24; then one rounding to bf16 (2^-8).  A sigmoid below 2^-126, where
    1 + e^-g or its reciprocal leaves FP32's normal range, becomes 0: that is off
    by less than 2^-126, and the output by less than 2^-126 |g u|; likewise an h
    below 2^-126 itself."""
    I = y.shape[1] // 2
    g, u = y[:, :I].astype(F64), y[:, I:].astype(F64)
    with np.errstate(over="ignore"):
        h = g / (1.0 + np.exp(-g)) * u
    return h, np.abs(h) * (2.0 ** -8 * 1.001 + (np.abs(g) + 8) * 2.0 ** -22) \
        + 2.0 ** -126 * (1 + np.abs(g * u))
