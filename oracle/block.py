"""CPU oracle of the block in 8 bits and of what stands around it: block-scaled e4m3 rows, the RMS norm
with the residual's addition, products by expert, dropout.  TEST INFRASTRUCTURE ONLY (see
``oracle.moe``).

Plain float64 numpy, written from the definitions.  Nothing is rounded but what the definitions round:
8-bit values (``e4m3_round``).  ``tests/test_block_oracle.py`` pins it: the gradients to central
differences, the formats to their tables, the generator to its authors' test vectors.
"""
from __future__ import annotations

import numpy as np

__all__ = ["BLOCK", "pitch", "e4m3_values", "e4m3_round", "scale_exponents", "quantize", "decode", "swiglu",
           "rms_norm", "rms_norm_backward", "grouped_gemm", "grouped_gemm_backward", "philox", "keep"]

BLOCK = 32


def pitch(cols):
    return 16 * -(-cols // 512)


def e4m3_values():
    """The 256 values of e4m3: sign, 4 exponent bits of bias 7, 3 fraction bits; 0x7f and 0xff NaN."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(b & 0x7F == 0x7F, np.nan, v)
    return np.where(b >= 128, -v, v)


def e4m3_round(v):
    """The nearest e4m3 values (ties to the even one) of values of at most 448 in magnitude."""
    v = np.asarray(v, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.abs(v))), -6)
    e = np.where(np.isfinite(e), e, -6)
    step = 2.0 ** (e - 3)
    return np.rint(v / step) * step


def scale_exponents(v):
    """For each block of 32 of the rows of v the smallest whole s >= -127 with max |v| <= 448 * 2^s."""
    v = np.asarray(v, np.float64)
    top = np.abs(np.where(np.isfinite(v), v, 0)).reshape(v.shape[0], v.shape[1] // BLOCK, BLOCK).max(-1)
    m, e = np.frexp(top)                                  # top = m 2^e, m in [1/2, 1)
    s = e - 9 + (m > 0.875)                               # 448 = 0.875 * 2^9
    return np.maximum(np.where(top == 0, -127, s), -127)


def quantize(v):
    """(values of the elements, scale bytes) of the rows of v; a value that is not finite is NaN."""
    v = np.asarray(v, np.float64)
    s = scale_exponents(v)
    x = np.where(np.isfinite(v), v, np.nan).reshape(*s.shape, BLOCK) / 2.0 ** s[..., None]
    bytes_ = np.zeros((v.shape[0], pitch(v.shape[1])), np.uint8)
    bytes_[:, :s.shape[1]] = s + 127
    return e4m3_round(x).reshape(v.shape), bytes_


def decode(q, scales):
    """The values that e4m3 bytes [rows][cols] and scale bytes [rows][pitch] stand for."""
    q, scales = np.asarray(q), np.asarray(scales)
    s = scales[:, :q.shape[1] // BLOCK].astype(np.float64) - 127
    return (e4m3_values()[q].reshape(q.shape[0], q.shape[1] // BLOCK, BLOCK) * 2.0 ** s[..., None]).reshape(q.shape)


def swiglu(x):
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    return g / (1 + np.exp(-g)) * u


def rms_norm(s, gamma, eps):
    """(y, rstd) of y[t] = s[t] * rstd_t * gamma."""
    s = np.asarray(s, np.float64)
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
    return s * rstd[:, None] * np.asarray(gamma, np.float64), rstd


def rms_norm_backward(dy, dsum, s, gamma, rstd):
    """(ds, dgamma) of rms_norm, with the statistic given and dsum reaching s past the norm."""
    dy, s, r = (np.asarray(t, np.float64) for t in (dy, s, rstd))
    xh = s * r[:, None]
    a = dy * np.asarray(gamma, np.float64)
    ds = r[:, None] * (a - xh * (a * xh).mean(axis=1)[:, None])
    return ds + (0 if dsum is None else np.asarray(dsum, np.float64)), (dy * xh).sum(axis=0)


def grouped_gemm(x, offsets, w):
    """y[r] = x[r] w[e]^T for the rows of each expert; w [E][N][K]."""
    y = np.zeros((x.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        y[rows] = x[rows] @ w[e].T
    return y


def grouped_gemm_backward(x, dy, offsets, w):
    """(dx, dw) of grouped_gemm."""
    dx, dw = np.zeros_like(x), np.zeros_like(w)
    for e in range(w.shape[0]):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        dx[rows] = dy[rows] @ w[e]
        dw[e] = dy[rows].T @ x[rows]
    return dx, dw


def philox(counter, key):
    """Philox4x32-10: counter four arrays of 32-bit words, key two; four arrays of words."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(w, np.uint64) for w in counter]
    k = [int(w) for w in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep(n, p, seed, step, first=0):
    """The mask of elements first .. first + n - 1."""
    i = np.arange(first, first + n, dtype=np.uint64)
    at = i // np.uint64(4)
    low = 0xFFFFFFFF
    words = philox((at & np.uint64(low), at >> np.uint64(32), np.full_like(at, step & low),
                    np.full_like(at, (step >> 32) & low)), (seed & low, (seed >> 32) & low))
    w = np.choose((i % np.uint64(4)).astype(np.int64), words)
    return w >= np.uint64(int(p * 2.0 ** 32))
