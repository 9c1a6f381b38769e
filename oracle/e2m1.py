"""Float64 NumPy oracle of rows held as OCP MX FP4 (E2M1 codes, a power-of-two
scale per 32 entries) and of the projection from them.  Written from the
definitions, to be checked by eye; it shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])  # by code, sign aside


def quantize(x: np.ndarray):
    """(codes [rows, cols], scale bytes [rows, cols / 32]) of float64 rows."""
    rows, cols = x.shape
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, cols // GROUP), np.uint8)
    for r in range(rows):
        for g in range(cols // GROUP):
            part = x[r, g * GROUP:(g + 1) * GROUP]
            if not np.isfinite(part).all():
                scales[r, g] = 255
                continue
            top = np.abs(part).max()
            e = 0
            if top > 0:
                e = -127
                while top > 7 * 2.0 ** e and e < 125:  # 6 * 2^126 is past fp32
                    e += 1
            scales[r, g] = e + 127
            for i, v in enumerate(part):
                off = np.abs(VALUES - abs(v) / 2.0 ** e)
                near = np.flatnonzero(off == off.min())
                code = near[0] if near[0] % 2 == 0 else near[-1]  # of two as near, the even one
                codes[r, g * GROUP + i] = code | (8 if np.signbit(v) else 0)
    return codes, scales


def pack(codes: np.ndarray) -> np.ndarray:
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What the codes stand for; NaN in groups of scale byte 255."""
    v = np.where(codes >= 8, -VALUES[codes & 7], VALUES[codes & 7])
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, GROUP, axis=1)


def logits(hidden: np.ndarray, codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return hidden @ values(codes, scales).T
