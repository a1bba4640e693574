"""Plain 64-bit references of the decode-step MoE layer and of the token
log-probabilities, with first-order bounds on the kernels' FP32 arithmetic."""
import numpy as np

U32 = 2.0 ** -24   # half a step of FP32
HALF = {"bf16": 2.0 ** -8, "f32": U32}  # half a step of the output type, relative
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3(b):
    b = b.astype(np.int64)
    e, m = b >> 3, (b & 7) / 8.0
    return np.where(e == 0, m * 2.0 ** -6, (1 + m) * 2.0 ** (e - 7.0))


def dequantize(codes, scales):
    """g * s_b (exact) of codes [N, K/2] and scales [N, K/16]."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    return E2M1[n] * np.repeat(e4m3(scales), 16, axis=1)


def route(logits, k):
    """(ids, weights): k largest logits, ties to the lower index, NaN as -inf."""
    lg = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    ids = np.argsort(-lg, axis=1, kind="stable")[:, :k]
    mx = lg.max(1, keepdims=True)
    mx = np.where(np.isinf(mx), 0.0, mx)
    p = np.exp(lg - mx)
    den = p.sum(1, keepdims=True)
    w = np.where(den > 0, p / np.where(den > 0, den, 1), 0.0)
    return ids.astype(np.int32), np.take_along_axis(w, ids, 1)


def moe_layer(x, logits, gu, down, k, dtype):
    """out [T, H] in 64 bits, and a bound on each value's error.

    gu, down: functions e -> (exact weights [N, K], tensor scale).  The
    bound: a product sum of n terms in FP32 is off by at most n U32 times the
    sum of the magnitudes; x and h enter with relative error r (one fp16
    piece: h by 2^-11, x exact; two pieces: 2^-21 for both, which leaves room for
    the second piece's own step) and what a power-of-two scale to the row's
    largest value loses below fp16's range, 2^-30 of that value; d silu <= 1.1;
    silu itself to 8 FP32 steps; the weights' exponentials to 2^-20."""
    T, H = x.shape
    ids, w = route(logits, k)
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    x = x.astype(np.float64)
    rx, rh = (0.0, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -21, 2.0 ** -21)
    for t in range(T):
        for s in range(k):
            if not w[t, s] > 0:
                continue
            wg, sg = gu(int(ids[t, s]))
            wd, sd = down(int(ids[t, s]))
            I = wd.shape[1]
            y = sg * (wg @ x[t])
            mag = sg * (np.abs(wg) @ np.abs(x[t]))
            dy = (H * U32 + rx) * mag + sg * 2.0 ** -30 * np.abs(x[t]).max() * np.abs(wg).sum(1) \
                + 2 * U32 * np.abs(y)
            g, u, dg, du = y[:I], y[I:], dy[:I], dy[I:]
            with np.errstate(over="ignore"):
                sl = g / (1 + np.exp(-g))
            h = sl * u
            dh = 1.1 * dg * np.abs(u) + (np.abs(sl) + 1.1 * dg) * du + 16 * U32 * np.abs(h)
            dh = dh + rh * (np.abs(h) + dh) + 2.0 ** -30 * np.abs(h).max()
            ww = w[t, s] * sd
            out[t] += ww * (wd @ h)
            tol[t] += ww * (np.abs(wd) @ (dh + (I + k + 4) * U32 * np.abs(h))) \
                + 2.0 ** -20 * np.abs(ww * (wd @ h))
    return ids, w, out, tol + HALF[dtype] * (np.abs(out) + tol) + 2.0 ** -133


def log_probs(logits, targets, inv_t, top_k):
    """dict of 64-bit logprobs, entropy, log p, top ids and values, and the
    bounds of their FP32 evaluation.

    2^d_j is off by U32 |d_j| from the argument (rounded once after a fused
    step; a further U32 |d_j| from the rounded factor c) and 2 U32 from the
    exponential; sums of up to V / 64 + 64 terms per chain add that many U32;
    log2 and the subtractions a few more."""
    z = logits.astype(np.float64)
    T, V = z.shape
    if inv_t is not None:
        z = z * inv_t.astype(np.float64)[:, None]
    m = z.max(1, keepdims=True)
    empty = np.isneginf(m[:, 0])
    with np.errstate(invalid="ignore", divide="ignore"):
        d = np.where(np.isneginf(z), -np.inf, z - np.where(empty[:, None], 0, m))
        s = np.exp(d).sum(1, keepdims=True)
        lp = np.where(np.isneginf(d), -np.inf, d - np.log(s))
    p = np.exp(lp)
    fin = np.where(np.isneginf(lp), 0.0, lp)
    df = np.where(np.isneginf(d), 0.0, d)
    ent = -(p * fin).sum(1)
    e1, e2 = (p * np.abs(df)).sum(1), (p * df * df).sum(1)
    chain = (V / 64 + 64) * U32
    dl = chain + 8 * U32 * (1 + e1)
    tol_lp = dl[:, None] + 8 * U32 * (1 + np.abs(fin) + np.abs(df))
    tol_h = chain * (1 + e1) + 8 * U32 * (1 + e1 + e2 + ent)
    r = dict(lp=lp, p=p, entropy=ent, tol_lp=tol_lp, tol_entropy=tol_h, empty=empty, lse=(
        np.where(empty, -np.inf, np.where(empty, 0, m[:, 0]) + np.log(np.where(empty, 1, s[:, 0])))))
    if targets is not None:
        at = np.take_along_axis(lp, np.clip(targets, 0, V - 1)[:, None], 1)[:, 0]
        r["logprobs"] = np.where(targets < 0, 0.0, np.where(targets >= V, np.nan, at))
        r["tol_logprobs"] = np.take_along_axis(tol_lp, np.clip(targets, 0, V - 1)[:, None], 1)[:, 0]
    if top_k:
        r["top_ids"] = np.argsort(-logits.astype(np.float64), axis=1, kind="stable")[:, :top_k]
        r["top_logprobs"] = np.take_along_axis(lp, r["top_ids"], 1)
        r["tol_top"] = np.take_along_axis(tol_lp, r["top_ids"], 1)
    return r


def log_probs_grad(r, targets, inv_t, ga, gb, dtype):
    """Gradient of the logits from log_probs's answer, and its bound."""
    p, lp = r["p"], np.where(np.isneginf(r["lp"]), 0.0, r["lp"])
    T, V = p.shape
    a = np.zeros(T) if ga is None else np.where((targets < 0) | r["empty"], 0.0, ga)
    b = np.zeros(T) if gb is None else gb.astype(np.float64)
    it = np.ones(T) if inv_t is None else inv_t.astype(np.float64)
    g = -p * (a[:, None] + b[:, None] * (lp + r["entropy"][:, None]))
    mag = p * (np.abs(a)[:, None] + np.abs(b)[:, None] * (np.abs(lp) + r["entropy"][:, None]))
    if ga is not None:
        rows = np.flatnonzero((targets >= 0) & (targets < V))
        g[rows, targets[rows]] += a[rows]
        mag[rows, targets[rows]] += np.abs(a[rows])
    # p is off by the error of log p, and the entropy's factor by its own
    tol = mag * (2 * r["tol_lp"] + 8 * U32) + np.abs(b)[:, None] * p * (
        r["tol_lp"] + r["tol_entropy"][:, None])
    g, tol = it[:, None] * g, it[:, None] * tol
    return g, tol + HALF[dtype] * (np.abs(g) + tol) + 2.0 ** -126
