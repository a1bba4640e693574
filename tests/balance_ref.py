"""Plain 64-bit reference of the router's balance loss and its gradient, with
tolerances derived from the operations.

u = 2^-24 is half a step of FP32.  With d = l - m the exponent of a
probability is off by three roundings relative to |d|, the exponential by two
steps, so e^d is off by (3 |d| + 4) u relative; their sum by the mean of that
and 16 additions; the reciprocal and the product add two roundings more:
p_j is off by dp_j = p_j (3 |d_j| + 3 D + 32) u with D = sum_j p_j |d_j|.
lse = m + ln s is off by that of s, a few steps of ln s and the last addition.
Sums over rows are FP32 over at most 512 rows and 64 bits above."""
import numpy as np

U = 2.0 ** -24


def balance(z, ids, mask=None, grad_losses=None, half_step=U):
    z = np.asarray(z, np.float64)
    T, E = z.shape
    k = ids.shape[1]
    live = ~(z == -np.inf).all(1)
    if mask is not None:
        live &= np.asarray(mask) != 0
    n = int(live.sum())
    zl, il = z[live], ids[live]
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        m = zl.max(1, keepdims=True, initial=-np.inf)
        d = zl - m
        e = np.exp(d)
        s = e.sum(1, keepdims=True)
        p = e / s
        lse = (m + np.log(s))[:, 0]
        ad = np.where(p > 0, np.abs(d), 0.0)
        D = (p * ad).sum(1, keepdims=True)
        dp = p * (3 * ad + 3 * D + 32) * U + 2.0 ** -125
        dlse = U * (np.abs(lse) + 4 * np.abs(np.log(s[:, 0])) + 3 * D[:, 0] + 32)
        inv = 1.0 / n if n else 0.0
        counts = np.bincount(il[(il >= 0) & (il < E)].astype(np.int64), minlength=E)
        P = p.sum(0) * inv
        dP = dp.sum(0) * inv + 516 * U * P
        f = E / k * inv * counts
        loss = (f * P).sum()
        zl2 = (lse ** 2).sum() * inv
        r = dict(counts=counts, tokens=n, mean_probs=P, tol_mean_probs=dP,
                 losses=np.array([loss, zl2]),
                 tol_losses=np.array([(f * dP).sum() + 4 * U * loss,
                                      (2 * np.abs(lse) * dlse).sum() * inv + 516 * U * zl2]))
        if grad_losses is None:
            return r
        a = float(grad_losses[0]) * E / k * inv * inv
        b = float(grad_losses[1]) * 2 * inv
        c = counts - counts.sum() / E
        cp = (p * c).sum(1, keepdims=True)
        dcp = (dp * np.abs(c)).sum(1, keepdims=True) + 18 * U * (p * np.abs(c)).sum(1, keepdims=True)
        fac = a * (c - cp) + b * lse[:, None]
        size = np.abs(a) * (np.abs(c) + np.abs(cp)) + np.abs(b * lse)[:, None]
        dfac = np.abs(a) * (dcp + U * np.abs(c)) + np.abs(b) * dlse[:, None] + 4 * U * size
        gl = p * fac
        tol = dp * np.abs(fac) + p * dfac + 2 * U * np.abs(gl)
        tol = tol + half_step * (np.abs(gl) + tol) + 2.0 ** -125
        grad, gtol = np.zeros((T, E)), np.zeros((T, E))
        grad[live], gtol[live] = gl, tol
        r.update(grad=grad, tol_grad=gtol)
    return r
