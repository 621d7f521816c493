"""8-bit blocks and the operators on them, in float64.

A block (128 consecutive features of a token, or a 128 x 128 piece of a weight; a last block may
be shorter) holds E4M3 codes and one scale 2^e: e is the smallest exponent >= -127 for which no
value exceeds 448 * 2^e, byte e + 127, byte 0 for a block of zeros. A block with an infinity or a
NaN has byte 0xFF and NaN codes. Where floating point decides a code, both sides decide in the
same precision: the norm's root is rounded to float32 and its two products are float32.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 128
NAN_CODE, NAN_SCALE = 0x7F, 0xFF


def _values() -> np.ndarray:
    """The 256 values of E4M3 (bias 7, no infinities, 0x7F and 0xFF NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = math.nan if (c & 0x7F) == NAN_CODE else (-v if c & 0x80 else v)
    return out


VALUES = _values()
_MAG = VALUES[:NAN_CODE]                                  # 0 .. 448, ascending
_MID = (_MAG[:-1] + _MAG[1:]) / 2


def codes_of(v) -> np.ndarray:
    """Nearest E4M3 code of each value in [-448, 448], ties to the even code."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    lo = np.searchsorted(_MID, a, side="left")            # a tie stays at the lower code
    tie = (lo < len(_MID)) & (a == _MID[np.minimum(lo, len(_MID) - 1)]) & (lo % 2 == 1)
    return ((lo + tie).astype(np.uint8) | (np.signbit(v).astype(np.uint8) << 7)).astype(np.uint8)


def exponent_of(amax: float) -> int:
    """Smallest e >= -127 with amax <= 448 * 2^e (amax > 0, finite)."""
    m, p = math.frexp(amax)
    return max(p - 9 + (m > 0.875), -127)


def _encode_block(b):
    if not np.all(np.isfinite(b)):
        return np.full(b.shape, NAN_CODE, np.uint8), NAN_SCALE
    top = float(np.max(np.abs(b)))
    e = exponent_of(top) if top > 0 else -127
    return codes_of(np.ldexp(b, -e)), e + 127


def encode_rows(X):
    """codes uint8 [M, K], scales uint8 [M, ceil(K / 128)]."""
    X = np.asarray(X, dtype=np.float64)
    M, K = X.shape
    codes, scales = np.empty((M, K), np.uint8), np.empty((M, -(-K // BLOCK)), np.uint8)
    for m in range(M):
        for j in range(scales.shape[1]):
            s = slice(j * BLOCK, min(K, (j + 1) * BLOCK))
            codes[m, s], scales[m, j] = _encode_block(X[m, s])
    return codes, scales


def encode_weight(W):
    """W [K, N] -> codes uint8 [N, K], scales uint8 [ceil(N / 128), ceil(K / 128)]."""
    Wt = np.asarray(W, dtype=np.float64).T
    N, K = Wt.shape
    codes, scales = np.empty((N, K), np.uint8), np.empty((-(-N // BLOCK), -(-K // BLOCK)), np.uint8)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.ix_(range(i * BLOCK, min(N, (i + 1) * BLOCK)), range(j * BLOCK, min(K, (j + 1) * BLOCK)))
            codes[at], scales[i, j] = _encode_block(Wt[at])
    return codes, scales


def _scale_values(scales):
    s = np.ldexp(1.0, scales.astype(int) - 127)
    return np.where(scales == NAN_SCALE, np.nan, s)


def decode_rows(codes, scales):
    return VALUES[codes] * np.repeat(_scale_values(scales), BLOCK, 1)[:, :codes.shape[1]]


def decode_weight(codes, scales):
    """[N, K] values."""
    s = np.repeat(np.repeat(_scale_values(scales), BLOCK, 0), BLOCK, 1)
    return VALUES[codes] * s[:codes.shape[0], :codes.shape[1]]


def rmsnorm(x, gamma, eps, residual=None, round_residual=None):
    """(y float32, updated residual): h = x + residual as one float32 sum rounded by
    round_residual, r = fp32(1 / sqrt(mean h^2 + eps)), y = (h r) gamma in float32 products."""
    h = np.asarray(x, dtype=np.float32)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float32)
        h = np.asarray(round_residual(h) if round_residual else h, dtype=np.float32)
    r = (1.0 / np.sqrt(np.mean(h.astype(np.float64) ** 2, axis=1, keepdims=True) + float(np.float32(eps))))
    y = (h * r.astype(np.float32)) * np.asarray(gamma, dtype=np.float32)
    return y, (h if residual is not None else None)


def activation(z, kind="silu"):
    z = np.asarray(z, dtype=np.float64)
    if kind == "silu":
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-z))
    return 0.5 * z * np.vectorize(math.erfc)(-z / math.sqrt(2.0))


def gated(A, Wg, Wu, kind="silu"):
    """A [M, K], Wg and Wu [N, K] decoded values."""
    return activation(A @ Wg.T, kind) * (A @ Wu.T)
