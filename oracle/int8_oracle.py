"""float64 oracle of the int8 quantizer and products and of the 16-bit experts' products with their
gradients, in NumPy from their definitions.  Shares no code with the HIP path."""
import numpy as np


def quantize(x):
    """Codes int8 [rows, cols] and scales float32 [rows] of float64 x holding bf16, fp16 or float32 values."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(x), x, 0.0)).max(1, initial=0.0))
    unit = np.where(amax > 0, amax, 1.0)
    # 127 x is exact; a quotient that is no border is at least 2^-33 from one, so float64 decides rightly
    q = np.rint(127.0 * np.where(bad[:, None], 0.0, x) / unit[:, None])
    scales = amax.astype(np.float32) / np.float32(127)
    scales[bad] = np.nan
    return q.astype(np.int8), scales


def dequantize(codes, scales):
    """float32 values (one rounding each)."""
    return codes.astype(np.float32) * scales.astype(np.float32)[:, None]


def product(a, sa, w, sw):
    """a [M, K], w [N, K] int8 with scales -> float64 [M, N]; the integer sums are exact in float64."""
    with np.errstate(invalid="ignore", over="ignore"):
        return (a.astype(np.float64) @ w.astype(np.float64).T) * sa.astype(np.float64)[:, None] * sw.astype(np.float64)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def grouped(x, w, offsets, counts, row_token=None):
    """{expert: (rows, y, sum of the products' magnitudes)} of y[r] = x[source(r)] @ w[e].T."""
    out = {}
    for e in np.nonzero(counts)[0]:
        r = np.arange(offsets[e], offsets[e] + counts[e])
        a = x[r if row_token is None else row_token[r]]
        out[e] = r, a @ w[e].T, np.abs(a) @ np.abs(w[e]).T
    return out


def grouped_grads(x, w, dy, offsets, counts, row_token=None):
    """{expert: (rows, dx, its magnitudes, dw, its magnitudes)}."""
    out = {}
    for e in np.nonzero(counts)[0]:
        r = np.arange(offsets[e], offsets[e] + counts[e])
        a, g = x[r if row_token is None else row_token[r]], dy[r]
        out[e] = r, g @ w[e], np.abs(g) @ np.abs(w[e]), g.T @ a, np.abs(g).T @ np.abs(a)
    return out
