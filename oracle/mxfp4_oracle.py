"""CPU oracle of the scored router and of the MXFP4 operators, in float64 NumPy from the definitions.

Independent of the HIP path: nothing here is used by the library.  MXFP4 (OCP microscaling): E2M1
elements, two per byte with the even element in the low nibble, one E8M0 scale (2**(byte - 127),
255 = NaN) per 32 consecutive elements.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x: np.ndarray):
    """codes uint8 [rows, cols/2] and scales uint8 [rows, cols/32] of float64 x [rows, cols]."""
    rows, cols = x.shape
    b = np.asarray(x, np.float64).reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 0.0, np.abs(b).max(-1))
    e = np.where(amax > 0, np.frexp(amax)[1] - 3, -127)  # frexp: amax = m * 2**(e+3), 0.5 <= m < 1
    e = np.maximum(e, -127)
    a = np.where(bad[..., None], 0.0, np.abs(b)) / np.ldexp(1.0, e)[..., None]
    mag = np.zeros(a.shape, np.uint8)
    for i in range(7):  # passes the midpoint of points i and i + 1; ties to the even code
        mid = (E2M1[i] + E2M1[i + 1]) / 2
        mag += ((a >= mid) if i % 2 else (a > mid)).astype(np.uint8)
    c = mag | (np.signbit(b).astype(np.uint8) << 3)
    c[bad] = 0
    c = c.reshape(rows, cols)
    return c[:, 0::2] | (c[:, 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of codes [..., K/2] and scales [..., K/32]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, -1)


def silu(g: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def product(a: np.ndarray, w: np.ndarray):
    """a [M, K] @ w [N, K]^T and the same of the magnitudes (for error bounds)."""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def gate_up(a: np.ndarray, w13: np.ndarray):
    """SiLU(gate) * up, and gate, up and the magnitudes' products of both."""
    z, zabs = product(a, w13)
    I = w13.shape[0] // 2
    return silu(z[:, :I]) * z[:, I:], z[:, :I], z[:, I:], zabs[:, :I], zabs[:, I:]


# ---- scored router -------------------------------------------------------------------------------

def finite_logits(logits: np.ndarray) -> np.ndarray:
    """float64 logits with NaN taken as -inf and +inf as the largest float32."""
    z = np.asarray(logits, np.float64)
    return np.where(np.isnan(z), -np.inf, np.minimum(z, float(np.finfo(np.float32).max)))


def shares(z: np.ndarray, kind: str) -> np.ndarray:
    """s_j / sum_i s_i of the scores of logits z [n], from their logarithms, which do not underflow
    (a softmax's common factor cancels); zeros where no logit is above -inf."""
    z = np.asarray(z, np.float64)
    if not np.any(z > -np.inf):
        return np.zeros(z.shape)
    log_s = -np.logaddexp(0.0, -z) if kind == "sigmoid" else z
    e = np.exp(log_s - log_s.max())
    return e / e.sum()


def scores(logits: np.ndarray, kind: str) -> np.ndarray:
    z = finite_logits(logits)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        m = z.max(1, keepdims=True)
        p = np.where(np.isneginf(z), 0.0, np.exp(z - np.where(np.isneginf(m), 0.0, m)))
        s = p.sum(1, keepdims=True)
        return np.where(s > 0, p / np.where(s > 0, s, 1.0), 0.0)


def router(logits, k, bias=None, score="sigmoid", n_group=1, topk_group=1, group_top=2, renormalize=True, scale=1.0):
    """ids int32 [T, k] (-1: none available) and weights float64 [T, k], one token at a time."""
    z, s = finite_logits(logits), scores(logits, score)
    T, E = s.shape
    c = s.astype(np.float32)
    if bias is not None:
        with np.errstate(invalid="ignore"):
            c = c + np.asarray(bias, np.float32)
    dead = ~(np.asarray(logits, np.float64) > -np.inf) | ~(c > -np.inf)
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    size = E // n_group
    for t in range(T):
        live = [e for e in range(E) if not dead[t, e]]
        if topk_group < n_group:
            by_group = []
            for g in range(n_group):
                best = sorted((c[t, e] for e in live if e // size == g), reverse=True)[:group_top]
                with np.errstate(over="ignore"):
                    total = np.float32(0) if not best else best[0] if len(best) == 1 else np.float32(best[0] + best[1])
                by_group.append((not best, -total, g))  # groups without an available expert come last
            kept = {g for *_, g in sorted(by_group)[:topk_group]}
            live = [e for e in live if e // size in kept]
        win = sorted(live, key=lambda e: (-c[t, e], e))[:k]
        ids[t, :len(win)] = win
        w[t, :len(win)] = scale * (shares(z[t, win], score) if renormalize else s[t, win])
    return ids, w


def router_bwd(logits, ids, grad, score="sigmoid", renormalize=True, scale=1.0):
    """Gradient of the weights with respect to the logits, float64 [T, E].  Renormalised, with
    n_j = s_j / S: dw_j / dz_e = scale n_j ([e = e_j] - n_e) f_e, f = 1 - s for sigmoid scores and 1 for
    softmax, whose sum over all experts cancels in n."""
    z, s = finite_logits(logits), scores(logits, score)
    out = np.zeros_like(s)
    for t in range(s.shape[0]):
        at = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < s.shape[1]]
        if not at:
            continue
        g = np.array([float(grad[t, j]) for j, _ in at])
        if renormalize:
            n = shares(z[t, [e for _, e in at]], score)
            part = scale * n * (n * (g[:, None] - g)).sum(1)  # n_j (g_j - sum_i n_i g_i), as a sum of what does not cancel
        else:
            part = scale * g
            if score == "softmax":  # s_e (G_e - sum_i s_i G_i), as a sum of what does not cancel
                G = np.zeros(s.shape[1])
                np.add.at(G, [e for _, e in at], part)
                out[t] = s[t] * (s[t] * (G[:, None] - G)).sum(1)
                continue
            part = part * s[t, [e for _, e in at]]
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                part = part / (1 + np.exp(z[t, [e for _, e in at]]))  # 1 - s, without the loss of a subtraction
        np.add.at(out[t], [e for _, e in at], part)
    return out
