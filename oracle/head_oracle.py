"""Float64 NumPy oracle of the low-precision linear layer's operators and of
the preference loss: microscaled quantisation, its products and gradients,
and the loss of paired log ratios with its gradient.  Plain definitions; it
shares no code with the HIP path."""

from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# OCP E4M3 magnitudes by code; code 127 is NaN
E4M3 = np.array([(f / 8.0) * 2.0 ** -6 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for f in range(8)][:127])


def ld(cols: int) -> int:
    return -(-cols // 128) * 128


def nearest_even(a: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the table value nearest to a (0 <= a <= table[-1]); a tie goes
    to the even index, which is the even last bit of the code."""
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    below, above = a - table[lo], table[hi] - a  # exact for these formats' values
    return np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))


def quantize(x: np.ndarray, fmt: str):
    """(codes, scales) of a float matrix, as include/casgd.h lays them out."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    table = E2M1 if fmt == "mx4" else E4M3
    b = np.zeros((rows, ld(cols)))
    b[:, :cols] = x
    b = b.reshape(rows, -1, 32)
    codes = np.zeros(b.shape, np.uint8)
    scales = np.full(b.shape[:2], 255, np.uint8)
    fine = np.isfinite(b).all(2)
    top = np.where(fine, np.abs(np.where(np.isfinite(b), b, 0)).max(2), 0.0)
    m, e = np.frexp(top / table[-1])  # top / largest = m 2^e, m in [1/2, 1): 2^(e - 1) only if m = 1/2
    byte = np.where(top > 0, e - (m == 0.5), -126) + 127
    byte = np.clip(byte, 1, 254)
    scales[fine] = byte[fine]
    u = b[fine] / (2.0 ** (byte[fine].astype(np.float64) - 127))[:, None]
    c = nearest_even(np.abs(u), table).astype(np.uint8)
    codes[fine] = c + np.where(np.signbit(u), 8 if fmt == "mx4" else 128, 0).astype(np.uint8)
    codes = codes.reshape(rows, -1)
    if fmt == "mx4":
        codes = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return codes, scales


def dequantize(codes: np.ndarray, scales: np.ndarray, cols: int, fmt: str) -> np.ndarray:
    if fmt == "mx4":
        c = np.empty((codes.shape[0], codes.shape[1] * 2), np.uint8)
        c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
        v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    else:
        v = np.where(codes >= 128, -1.0, 1.0) * np.append(E4M3, np.nan)[codes & 127]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v.reshape(v.shape[0], -1, 32) * s[:, :, None]).reshape(v.shape)[:, :cols]


def rounded(x, fmt: str) -> np.ndarray:
    codes, scales = quantize(x, fmt)
    return dequantize(codes, scales, np.shape(x)[1], fmt)


def token_logps(z: np.ndarray, labels: np.ndarray) -> np.ndarray:
    out = np.zeros(len(z))
    for t, y in enumerate(labels):
        if y >= 0:
            m = z[t].max()
            out[t] = z[t][y] - m - np.log(np.exp(z[t] - m).sum())
    return out


def pair_loss(h: float, kind: str, beta: float, eps: float):
    """(loss, derivative in h)."""
    if kind == "logistic":
        u = beta * h
        plus = np.logaddexp(0.0, u)    # log(1 + exp(u))
        minus = np.logaddexp(0.0, -u)
        return (1 - eps) * minus + eps * plus, beta * (eps - np.exp(-plus))
    r = h - 0.5 / beta
    return r * r, 2 * r


def preference(z, labels, offsets, ref, beta, kind="logistic", eps=0.0, average=False, grad_loss=None):
    """dict of loss, margin, logps, slope (per sequence) and, with grad_loss, dlogits."""
    z = np.asarray(z, np.float64)
    lp = token_logps(z, labels)
    pairs = (len(offsets) - 1) // 2
    ref = np.zeros(len(z)) if ref is None else np.asarray(ref, np.float64)
    loss, margin, slope = np.zeros(pairs), np.zeros(pairs), np.zeros(2 * pairs)
    d = np.zeros_like(z)
    for p in range(pairs):
        share, total = [], []
        for side in (0, 1):
            a, b = offsets[2 * p + side], offsets[2 * p + side + 1]
            rows = [t for t in range(a, b) if labels[t] >= 0]
            share.append(1.0 / len(rows) if average and rows else 1.0)
            total.append(sum(lp[t] - ref[t] for t in rows) * share[-1])
        margin[p] = total[0] - total[1]
        loss[p], g = pair_loss(margin[p], kind, beta, eps)
        slope[2 * p], slope[2 * p + 1] = g * share[0], -g * share[1]
        if grad_loss is None:
            continue
        for side in (0, 1):
            for t in range(offsets[2 * p + side], offsets[2 * p + side + 1]):
                if labels[t] < 0:
                    continue
                m = z[t].max()
                q = np.exp(z[t] - m)
                row = -q / q.sum()
                row[labels[t]] += 1
                d[t] = slope[2 * p + side] * grad_loss[p] * row
    return {"loss": loss, "margin": margin, "logps": lp, "slope": slope, "dlogits": d}
