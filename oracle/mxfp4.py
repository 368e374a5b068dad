"""MXFP4 rows: E2M1 elements with one E8M0 scale per 32 of them.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Definition: include/nvfp4_moe.h, "MXFP4 rows".  Pinned by ``tests/test_oracle_mxfp4.py``.
"""

import numpy as np

from .formats import e2m1_decode, e2m1_encode

BLOCK = 32


def quantize_rows(x):
    """x [rows, C] (FP32 values, C % 32 == 0) -> (codes uint8 [rows, C], scales uint8 [rows, C/32])."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    b = x.reshape(rows, cols // BLOCK, BLOCK).astype(np.float64)
    bad = ~np.isfinite(b).all(-1)
    top = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)
    scale = np.clip(e + 127, 0, 254)
    with np.errstate(invalid="ignore"):
        q = b / np.exp2(scale - 127.0)[..., None]          # exact: a power of two
    codes = np.where(bad[..., None], 0, e2m1_encode(np.where(bad[..., None], 0.0, q)))
    return codes.astype(np.uint8).reshape(rows, cols), np.where(bad, 255, scale).astype(np.uint8)


def dequantize_rows(codes, scales):
    """FP64 values; a scale of 255 gives NaN."""
    codes = np.asarray(codes, np.uint8)
    rows, cols = codes.shape
    s = np.where(scales == 255, np.nan, np.exp2(np.asarray(scales, np.float64) - 127.0))
    return (e2m1_decode(codes).reshape(rows, cols // BLOCK, BLOCK) * s[..., None]).reshape(rows, cols)


def sf_byte_index(rows, cols):
    """[rows, cols/32] byte of each scale in the 512-byte tiles."""
    r = np.arange(rows)[:, None]
    b = np.arange(cols // BLOCK)[None, :]
    return ((r // 128) * -(-cols // 128) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
