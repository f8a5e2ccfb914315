"""Plain CPU oracle of the experts' steps (test infrastructure only).

NumPy in 64 bits, straight from the definitions in ``include/ultraep_experts.h``:
the e4m3 block format, the grouped products, the weight gradients and the
clipping.  Shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def e4m3_values() -> np.ndarray:
    """The 256 values of OCP e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        mag = (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        v[b] = -mag if b & 128 else mag
    v[0x7F] = v[0xFF] = np.nan
    return v


VALUES = e4m3_values()
_GRID = VALUES[:0x7F]  # the finite magnitudes, ascending; a byte's last bit is its mantissa's


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 byte of values of magnitude at most 448 (ties to the even mantissa); others: NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    ok = a <= 448.0
    a = np.where(ok, a, 0.0)
    hi = np.minimum(np.searchsorted(_GRID, a, side="left"), 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    out = np.where(ok, pick, 0x7F).astype(np.uint8)
    return out | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)


def block_exponent(x: np.ndarray, axes) -> np.ndarray:
    """Smallest e >= -126 with the block's largest finite magnitude <= 448 * 2^e; 0 for a block of zeros."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(axis=axes)
    e = np.full(a.shape, -126)
    for k in range(-126, 130):
        e = np.where(a > 448.0 * 2.0 ** k, k + 1, e)
    return np.where(a == 0, 0, e)


def up(n: int, m: int = BLOCK) -> int:
    return -(-n // m) * m


def quant_rows(x: np.ndarray):
    """Rows form (q, scale) of [rows, H]."""
    rows, H = x.shape
    kb = up(H) // BLOCK
    g = np.zeros((rows, kb * BLOCK))
    g[:, :H] = x
    g = g.reshape(rows, kb, BLOCK)
    e = block_exponent(g, 2)
    scale = np.full((rows, up(kb, 4)), 127, dtype=np.uint8)
    scale[:, :kb] = e + 127
    return to_e4m3(g / 2.0 ** e[:, :, None]).reshape(rows, kb * BLOCK), scale


def first_blocks(off) -> list:
    return [int(o) // BLOCK + p for p, o in enumerate(off)]


def quant_cols(x: np.ndarray, off, blocks: int, fill: int = 0):
    """Columns form (qt, scale) of [rows, H] with expert offsets off; blocks without an expert hold `fill`."""
    H = x.shape[1]
    qt = np.full((blocks, H, BLOCK), fill, dtype=np.uint8)
    scale = np.full((blocks, H), fill, dtype=np.uint8)
    for p, b in enumerate(first_blocks(off)[:-1]):
        for i, at in enumerate(range(off[p], off[p + 1], BLOCK)):
            g = np.zeros((BLOCK, H))
            part = x[at:min(at + BLOCK, off[p + 1])]
            g[:len(part)] = part
            e = block_exponent(g, 0)
            qt[b + i] = to_e4m3(g / 2.0 ** e).T
            scale[b + i] = e + 127
    return qt, scale


def quant_weight(w: np.ndarray):
    """Weights form (q, scale) of [N, K]."""
    N, K = w.shape
    nb, kb = up(N) // BLOCK, up(K) // BLOCK
    g = np.zeros((nb * BLOCK, kb * BLOCK))
    g[:N, :K] = w
    g = g.reshape(nb, BLOCK, kb, BLOCK)
    e = block_exponent(g, (1, 3))
    scale = np.full((nb, up(kb, 4)), 127, dtype=np.uint8)
    scale[:, :kb] = e + 127
    return to_e4m3(g / 2.0 ** e[:, None, :, None]).reshape(nb * BLOCK, kb * BLOCK)[:N], scale


def rows_value(q: np.ndarray, scale: np.ndarray) -> np.ndarray:
    kb = q.shape[1] // BLOCK
    return VALUES[q] * np.repeat(2.0 ** (scale[:, :kb].astype(np.float64) - 127), BLOCK, axis=1)


def weight_value(q: np.ndarray, scale: np.ndarray) -> np.ndarray:
    return rows_value(q, np.repeat(scale, BLOCK, axis=0)[:q.shape[0]])


def expert_gemm(x: np.ndarray, w: list, off) -> np.ndarray:
    """x [rows, K'], w: per expert [N, K'] (both dequantised)."""
    return np.concatenate([x[off[p]:off[p + 1]] @ w[p].T for p in range(len(w))])


def expert_wgrad(dyt, dyt_scale, xt, xt_scale, off) -> list:
    """Per expert sum over its rows of dy x^T, from the columns forms."""
    out = []
    for p, b in enumerate(first_blocks(off)[:-1]):
        n = -(-(off[p + 1] - off[p]) // BLOCK)
        g = np.zeros((dyt.shape[1], xt.shape[1]))
        for i in range(b, b + n):
            dy = VALUES[dyt[i]] * 2.0 ** (dyt_scale[i].astype(np.float64) - 127)[:, None]
            x = VALUES[xt[i]] * 2.0 ** (xt_scale[i].astype(np.float64) - 127)[:, None]
            g += dy @ x.T
        out.append(g)
    return out


def clip(tensors: list, max_norm: float):
    """(norm, clipped tensors) in 64 bits."""
    norm = float(np.sqrt(sum(float(np.sum(np.square(t, dtype=np.float64))) for t in tensors)))
    c = min(1.0, max_norm / (norm + 1e-6))
    return norm, [t.astype(np.float64) * c for t in tensors]
