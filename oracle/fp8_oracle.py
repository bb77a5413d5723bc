"""float64 reference of the 8-bit operators (numpy), written from their
formulas: e4m3 codes with one scale per 128 values, the RMS norm with the
residual's addition, the gated activation and the scaled product.

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; exponent field 0 is
subnormal (m / 8 * 2^-6); field 15 is an ordinary binade except mantissa 7,
which is NaN.  Largest value 448.
"""
from __future__ import annotations

import numpy as np

RUN = 128
MAX = 448.0
MIN_SCALE = 2.0 ** -126


def _table() -> np.ndarray:
    v = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        mag = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            mag = np.nan
        v[code] = -mag if code & 128 else mag
    return v


VALUES = _table()


def decode(codes: np.ndarray) -> np.ndarray:
    """Values of uint8 codes."""
    return VALUES[codes]


def encode(v: np.ndarray) -> np.ndarray:
    """uint8 codes of values, nearest, ties to the even code; |v| <= 448 after rounding."""
    v = np.asarray(v, dtype=np.float64)
    pos = VALUES[:127]                      # 0 .. 448, increasing
    mag = np.minimum(np.abs(v), MAX)
    hi = np.clip(np.searchsorted(pos, np.nan_to_num(mag)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = mag - pos[lo], pos[hi] - mag
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(np.isnan(v), 127, code)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def runs(n: int) -> int:
    return -(-n // RUN)


def row_scales(v: np.ndarray) -> np.ndarray:
    """[M][ceil(D/128)] scales of the rows of v."""
    M, D = v.shape
    out = np.empty((M, runs(D)))
    for b in range(runs(D)):
        out[:, b] = np.maximum(np.abs(v[:, b * RUN:(b + 1) * RUN]).max(axis=1) / MAX, MIN_SCALE)
    return out


def spread(scales: np.ndarray, D: int) -> np.ndarray:
    """Row scales repeated to [M][D]."""
    return np.repeat(scales, RUN, axis=1)[:, :D]


def code_rows(v: np.ndarray):
    s = row_scales(v).astype(np.float32)
    return encode(v / spread(s.astype(np.float64), v.shape[1])), s


def code_weight(w: np.ndarray):
    N, K = w.shape
    s = np.empty((runs(N), runs(K)), dtype=np.float32)
    for i in range(runs(N)):
        for j in range(runs(K)):
            blk = np.abs(w[i * RUN:(i + 1) * RUN, j * RUN:(j + 1) * RUN])
            s[i, j] = max(blk.max() / MAX, MIN_SCALE)
    full = np.repeat(np.repeat(s.astype(np.float64), RUN, axis=0), RUN, axis=1)[:N, :K]
    return encode(w / full), s


def rmsnorm(x, residual, w, eps):
    """(h, y) in float64."""
    h = x if residual is None else x + residual
    return h, h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * w


def silu_mul(gate_up):
    D = gate_up.shape[1] // 2
    g, u = gate_up[:, :D], gate_up[:, D:]
    return g / (1 + np.exp(-g)) * u


def product(a, sa, w, sw):
    """(y, sum of the magnitudes of its terms) for codes a [M][K], w [N][K]."""
    K, N = a.shape[1], w.shape[0]
    av = decode(a) * spread(sa.astype(np.float64), K)
    wv = decode(w) * np.repeat(spread(sw.astype(np.float64), K), RUN, axis=0)[:N]
    return av @ wv.T, np.abs(av) @ np.abs(wv).T
