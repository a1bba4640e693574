"""The decode-step MoE layer in 64 bits for large sizes, expert by expert in
torch on any device, with the error bound of decode_ref.moe_layer but for the
length of the FP32 sums.

A product sum of K terms is not one chain of K roundings.  A term goes through
at most one MFMA of 32 terms, the 16 that follow it in a K range (512 k, or 256
k of FP32's two pieces), the ranges, and the waves that share K.  Counted as
one whole step each (2 U32), since the order and rounding inside an MFMA are
the hardware's: (2 (32 + 16) + K / 256 + 8) U32 of the summed magnitudes."""
import torch

import decode_ref as R

U32 = R.U32
E2M1 = torch.tensor(R.E2M1)


def dequantize(codes, scales):
    """decode_ref.dequantize of device tensors."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(1).long()
    b = scales.long()
    e, m = b >> 3, (b & 7).double() / 8
    s = torch.where(e == 0, m * 2.0 ** -6, torch.ldexp(1 + m, e - 7))
    return E2M1.to(codes.device)[n] * s.repeat_interleave(16, 1)


def chain(K):
    return (2 * (32 + 16) + K / 256 + 8) * U32


def moe_layer(x, logits, gu, down, k, dtype, chain=chain):
    """(ids, weights, out, tol) of x [T, H] and logits [T, E]; gu and down are
    (codes [E, N, K/2], scales [E, N, K/16], tensor scales [E])."""
    ids, w = R.route(logits.cpu().numpy(), k)
    x = x.double()
    T, H = x.shape
    I = down[0].shape[2] * 2
    out, tol = torch.zeros_like(x), torch.zeros_like(x)
    rx, rh = (0.0, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -21, 2.0 ** -21)
    for e in sorted(set(ids[w > 0].tolist())):
        t, s = (torch.from_numpy(i).to(x.device) for i in ((ids == e) & (w > 0)).nonzero())
        ww = torch.from_numpy(w).to(x.device)[t, s][:, None] * float(down[2][e])
        sg = float(gu[2][e])
        wg = dequantize(gu[0][e], gu[1][e]).T.contiguous()
        y = sg * (x[t] @ wg)
        wg.abs_()
        mag = sg * (x[t].abs() @ wg)
        dy = (chain(H) + rx) * mag + sg * 2.0 ** -30 * x[t].abs().amax(1, keepdim=True) * wg.sum(0) \
            + 2 * U32 * y.abs()
        del wg
        g, u, dg, du = y[:, :I], y[:, I:], dy[:, :I], dy[:, I:]
        sl = g * torch.sigmoid(g)
        h = sl * u
        dh = 1.1 * dg * u.abs() + (sl.abs() + 1.1 * dg) * du + 16 * U32 * h.abs()
        dh = dh + rh * (h.abs() + dh) + 2.0 ** -30 * h.abs().amax(1, keepdim=True)
        wd = dequantize(down[0][e], down[1][e]).T.contiguous()
        part = ww * (h @ wd)
        out.index_add_(0, t, part)
        wd.abs_()
        tol.index_add_(0, t, ww * ((dh + (chain(I) + (k + 4) * U32) * h.abs()) @ wd)
                       + 2.0 ** -20 * part.abs())
    return ids, w, out, tol + R.HALF[dtype] * (out.abs() + tol) + 2.0 ** -133
