"""Block-128 FP8: the quantizer, the products and the expert of FT_FP8, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

* A block (1 x 128 elements of a row, or 128 x 128 of a matrix; the last ones
  partial) shares the scale 2^max(-126, ceil(log2(amax / 448))), the smallest
  power of two that brings it within E4M3; a code is the E4M3 value nearest to
  the quotient, ties to the even code.  A block with a NaN or an infinity has
  scale NaN and codes 0.
* An element is its E4M3 value (``mx.e4m3_to_f64``) times its block's scale.
* The expert quantizes x and the SwiGLU hidden vector by 1 x 128 blocks.
"""
from __future__ import annotations

import numpy as np

from .mx import e4m3_to_f64, round_to_e4m3

BLOCK = 128
E4M3_MAX = 448.0


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def block_max(v: np.ndarray, block_rows: int) -> np.ndarray:
    """Largest magnitude of each block (NaN where the block holds a NaN)."""
    n, K = v.shape
    nb = -(-n // block_rows)
    a = np.zeros((nb * block_rows, _blocks(K) * BLOCK))
    a[:n, :K] = np.abs(v)
    return a.reshape(nb, block_rows, _blocks(K), BLOCK).max(axis=(1, 3))


def scale_of(amax: np.ndarray) -> np.ndarray:
    """The block scale of a largest magnitude, from its exact binary form."""
    amax = np.asarray(amax, np.float64)
    with np.errstate(invalid="ignore"):
        f, p = np.frexp(np.where(np.isfinite(amax), amax, 1.0))      # amax = f 2^p, f in [0.5, 1); 448 = 0.875 2^9
    e = np.where(f <= 0.875, p - 9, p - 8)
    e = np.where(amax == 0, -126, np.maximum(e, -126))
    return np.where(np.isfinite(amax), np.ldexp(1.0, e), np.nan)


def spread(scales: np.ndarray, block_rows: int, n: int, K: int) -> np.ndarray:
    """Block scales -> one per element [n, K]."""
    return np.repeat(np.repeat(scales, block_rows, axis=0)[:n], BLOCK, axis=1)[:, :K]


def quantize(v: np.ndarray, block_rows: int = 1) -> tuple[np.ndarray, np.ndarray]:
    """v [n, K] -> codes [n, K] uint8, scales [ceil(n / block_rows), ceil(K / 128)] float64."""
    v = np.asarray(v, np.float64)
    s = scale_of(block_max(v, block_rows))
    S = spread(s, block_rows, *v.shape)
    ok = np.isfinite(S)
    codes = round_to_e4m3(np.where(ok, v, 0.0) / np.where(ok, S, 1.0))
    return np.where(ok, codes, 0).astype(np.uint8), s


def to_f64(codes: np.ndarray, scales: np.ndarray, block_rows: int = 1) -> np.ndarray:
    """Codes and scales -> the float64 values they stand for."""
    codes = np.asarray(codes, np.uint8)
    n, K = codes.shape
    scales = np.asarray(scales, np.float64)
    if scales.shape != (-(-n // block_rows), _blocks(K)):
        raise ValueError("scale array does not match the code array")
    return e4m3_to_f64(codes) * spread(scales, block_rows, n, K)


def swiglu_expert(x: np.ndarray, wg, wu, wd) -> np.ndarray:
    """One FP8 expert on rows x [n, H] (float64): x and h go through the quantizer."""
    xq = to_f64(*quantize(x))
    g, u = xq @ wg.T, xq @ wu.T
    h = g / (1.0 + np.exp(-g)) * u
    return to_f64(*quantize(h)) @ wd.T
