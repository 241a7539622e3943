"""Float64 CPU oracle of the 4-bit key/value cache: rounding, storing, reading back, and
attention over the values the cache stands for.

TEST INFRASTRUCTURE ONLY, as ``oracle.attention``; it shares no code with the CUDA library.

Each rounding is written as a search for the nearest of all representable values, in float64:

* scale    the values of 5 exponent bits (bias 15) and 3 mantissa bits up to 10240, byte by byte;
           s is the one nearest to max|x| / 6 (a tie goes to the even byte), 255 for a NaN;
* element  0, .5, 1, 1.5, 2, 3, 4, 6 (codes 0 to 7); the one nearest to |x| / s (a tie goes to the
           even code), the sign in bit 3; 0 where s = 0 or the block has a NaN.

The quotients of float32 inputs are exact enough in float64: they differ from a midpoint by at
least 2^-24 relative or not at all, and a quotient that is a midpoint has at most 6 significant
bits, so its float64 value is exact.
"""

from __future__ import annotations

import numpy as np

from . import attention as orc

BLOCK = 16
SCALES = np.array([b * 2.0 ** -17 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 15) for b in range(227)])
ELEMENTS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nearest(grid: np.ndarray, x: np.ndarray) -> np.ndarray:
    """Index of the value of the ascending grid nearest to x; the even index at a tie."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo = np.searchsorted(mid, x, side="left")
    hi = np.searchsorted(mid, x, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def quantise(x: np.ndarray):
    """(codes, scales) of rows x (..., E) float64: uint8 arrays (..., E/2) and (..., E/16)."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (-1, BLOCK))
    nan = np.isnan(b).any(-1)
    most = np.abs(np.where(np.isnan(b), 0.0, b)).max(-1)
    byte = nearest(SCALES, most / 6.0)
    s = np.where(nan, 0.0, SCALES[byte])[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        code = nearest(ELEMENTS, np.where(s > 0, np.abs(b) / s, 0.0))
    code = np.where(s > 0, code | (np.signbit(b).astype(np.int64) << 3), 0)
    code = code.reshape(x.shape)
    return ((code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8),
            np.where(nan, 255, byte).astype(np.uint8))


def dequantise(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The float64 values (..., E) of cache bytes (NaN for the scale byte 255)."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1, BLOCK))
    table = np.concatenate([SCALES, np.full(256 - len(SCALES), np.nan)])
    v = np.where(c & 8, -ELEMENTS[c & 7], ELEMENTS[c & 7]) * table[scales][..., None]
    return v.reshape(codes.shape[:-1] + (-1,))


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, lens, *, scale: float, mode: str = "dot", sink=None,
              mask_kind: str = "none", window: int = 0, keep: int = 0):
    """Attention of q (N, Hq, L, E) over the first lens[n] rows of k (N, H, C, E), v (N, H, C, Ev), all float64."""
    N, Hq, L, _ = q.shape
    out = np.zeros((N, Hq, L, v.shape[-1]))
    lse = np.full((N, Hq, L), -np.inf)
    for n in range(N):
        if lens[n] == 0:
            if sink is not None:
                lse[n] = np.asarray(sink)[:, None]
            continue
        out[n:n + 1], lse[n:n + 1] = orc.attention_forward(
            q[n:n + 1], k[n:n + 1, :, :lens[n]], v[n:n + 1, :, :lens[n]], scale=scale, mode=mode, sink=sink,
            mask_kind=mask_kind, window=window, keep=keep)
    return out, lse
