"""Plain 64-bit reference of the 4-bit microscaled format and of the grouped-row operators."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x: np.ndarray):
    """(codes uint8 [n, ceil32(d)], scale bytes uint8 [n, blocks], values float64 [n, d])."""
    x = np.asarray(x, np.float64)
    n, d = x.shape
    blocks = -(-d // 32)
    xb = np.zeros((n, blocks * 32))
    xb[:, :d] = x
    xb = xb.reshape(n, blocks, 32)
    amax = np.abs(xb).max(2)
    bad = ~np.isfinite(xb).all(2)
    with np.errstate(all="ignore"):
        _, ex = np.frexp(np.where(bad, 1.0, amax))        # amax = m 2^ex, 0.5 <= m < 1
    e = np.where(amax > 0, np.clip(ex - 1 - 2, -127, 127), -127)
    a = np.abs(np.where(bad[:, :, None], 0.0, xb)) / np.exp2(e)[:, :, None]
    lo = np.searchsorted(LEVELS, a, side="right") - 1
    hi = np.minimum(lo + 1, 7)
    down, up = a - LEVELS[lo], LEVELS[hi] - a
    idx = np.where((up < down) | ((up == down) & (lo % 2 == 1)), hi, lo)
    sign = np.where(np.signbit(xb), 8, 0)
    codes = np.where(bad[:, :, None], 0, idx + sign).astype(np.uint8)
    values = np.where(np.signbit(xb), -1.0, 1.0) * LEVELS[idx] * np.exp2(e)[:, :, None]
    values[bad] = np.nan
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes.reshape(n, -1), scale, values.reshape(n, -1)[:, :d]


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def tile_scales(scale: np.ndarray) -> np.ndarray:
    """Scale bytes [n, blocks] -> tiles [ceil(n/128), 2 ceil(blocks/8), 32, 4, 4], zeros elsewhere."""
    n, blocks = scale.shape
    out = np.zeros((-(-n // 128), 2 * -(-blocks // 8), 32, 4, 4), np.uint8)
    r, b = np.meshgrid(np.arange(n), np.arange(blocks), indexing="ij")
    out[r // 128, b // 4, r % 32, r % 128 // 32, b % 4] = scale
    return out


def group(row_slots: np.ndarray, n_slots: int):
    """(offsets, slots, order, positions) as mlora_group_rows defines them."""
    flat = np.asarray(row_slots).reshape(-1)
    N = flat.size
    S = min(n_slots + 1, N)
    valid = (flat >= -1) & (flat < n_slots)
    key = np.where(valid, flat, n_slots)
    order = np.argsort(key, kind="stable")
    positions = np.empty(N, np.int64)
    positions[order] = np.arange(N)
    positions[~valid] = -1
    used = np.unique(flat[valid])
    slots = np.full(S, -1)
    slots[:used.size] = used
    offsets = np.full(S + 1, int(valid.sum()))
    offsets[0] = 0
    for g, a in enumerate(used):
        offsets[g + 1] = offsets[g] + int((flat == a).sum())
    return offsets, slots, order, positions
