"""8-bit activation checkpoints in fp64 (oracle).

Test infrastructure: only the tests may use this module.

A block is 64 consecutive values of a row of bf16 activations; with ``a`` its
absolute maximum

* int8: ``step = bf16(a / 127)``, ``q = round(x / step)`` cut to [-127, 127];
* E4M3: ``step = bf16(a / 256)``, ``q = E4M3(x / step)``, saturating;

and the block stands for ``bf16(q step)``.  All roundings are to nearest even.
The int8 step is at most 2^121; a block with a NaN or an infinity has a NaN
step, and -0 has code 0.  Every intermediate here is an exact fp64 value or an fp64 quotient of
two 8-bit significands, which is nowhere near a rounding border unless it is
one exactly.
"""

from __future__ import annotations

import numpy as np

from .nf4 import e4m3_decode, e4m3_encode

BLOCK = 64


def round_bf16(v) -> np.ndarray:
    """fp64 -> the nearest bf16 value (as fp64), ties to even, subnormals and overflow included."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        _, e = np.frexp(v)
        unit = np.ldexp(1.0, np.maximum(e, -125) - 8)
        r = np.rint(v / unit) * unit
        r = np.where(np.abs(r) >= 2.0**128, np.sign(r) * np.inf, r)
    return np.where(np.isfinite(v), r, v)


def encode(x, fmt: str):
    """(codes uint8 [n], steps fp64 [n / 64]) of bf16 values x (any shape, as fp64)."""
    b = np.asarray(x, dtype=np.float64).reshape(-1, BLOCK)
    bad = ~np.isfinite(b).all(axis=1)
    b = np.where(bad[:, None], 0.0, b)
    step = round_bf16(np.abs(b).max(axis=1) / (127.0 if fmt == "int8" else 256.0))
    if fmt == "int8":
        step = np.minimum(step, 2.0**121)
    q = np.where(step[:, None] > 0, b / np.where(step > 0, step, 1.0)[:, None], 0.0) + 0.0  # -0 -> 0
    if fmt == "int8":
        codes = np.clip(np.rint(q), -127, 127).astype(np.int8).view(np.uint8)
    else:
        codes = e4m3_encode(q)
    return codes.ravel(), np.where(bad, np.nan, step)


def decode(codes, step, fmt: str) -> np.ndarray:
    """fp64 values (each a bf16 value) of codes [n] with steps [n / 64]."""
    c = np.asarray(codes, dtype=np.uint8)
    q = (c.view(np.int8) if fmt == "int8" else e4m3_decode(c)).astype(np.float64)
    with np.errstate(invalid="ignore"):
        return round_bf16(q.reshape(-1, BLOCK) * np.asarray(step, dtype=np.float64)[:, None]).ravel()
