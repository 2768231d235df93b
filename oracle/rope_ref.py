"""ORACLE (test infrastructure only): rotary positions and the KV write of a
ragged batch, in fp64, from the formulas of hpc_rope_init and
hpc_rope_kv_write in include/hpc_decode.h. Only tests/ may use it."""
from __future__ import annotations

import math
from typing import List, Tuple

import numpy as np


def frequencies(R: int, base: float, scaling: str = "none", factor: float = 1.0,
                original_len: int = 0, low: float = 0.0, high: float = 0.0) -> Tuple[np.ndarray, float]:
    """(angle per position of each pair, magnitude)."""
    if scaling == "base":
        base = base * factor ** (R / (R - 2))
    out: List[float] = []
    for i in range(R // 2):
        f = 1.0 / base ** (2 * i / R)
        if scaling == "linear":
            f = f / factor
        elif scaling == "banded":
            wavelength = 2 * math.pi / f
            if original_len / wavelength <= low:
                f = f / factor
            elif original_len / wavelength < high:
                w = (original_len / wavelength - low) / (high - low)
                f = w * f + (1 - w) * f / factor
        elif scaling == "ramp":
            index = lambda t: R * math.log(original_len / (2 * math.pi * t)) / (2 * math.log(base))
            a, b = max(0, math.floor(index(high))), min(R - 1, math.ceil(index(low)))
            u = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            f = u * f / factor + (1 - u) * f
        out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1 if scaling == "ramp" else 1.0)


def turn(x: np.ndarray, positions, freq: np.ndarray, magnitude: float, R: int,
         interleaved: bool) -> np.ndarray:
    """x [N][H][D] fp64; the first R elements of each row turned."""
    y = np.array(x, dtype=np.float64)
    for n, p in enumerate(positions):
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            c, s = magnitude * math.cos(int(p) * freq[i]), magnitude * math.sin(int(p) * freq[i])
            y[n, :, a] = x[n, :, a] * c - x[n, :, b] * s
            y[n, :, b] = x[n, :, b] * c + x[n, :, a] * s
    return y


def norm(x: np.ndarray, w, eps: float) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    if w is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)
