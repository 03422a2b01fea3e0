"""The operators around the grouped GEMM in 64 bits, written from their definitions on the CPU
(numpy and torch float64), and the check of a quantised operand against exact values.

A quantised element is right if it is the nearest code to v / s for some v within the stated
relative error u of the exact value (u = 0: exactly the nearest, ties to even), s being the scale that
was stored; a scale is right if it lies between the scales of amax * (1 - u) and amax * (1 + u).
"""
from __future__ import annotations

import numpy as np
import torch

VEC = {"blockwise": 128, "mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
TOP = {"blockwise": 448.0, "mxfp8": 448.0, "mxfp4": 6.0, "nvfp4": 6.0}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)]
                + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])
assert E4M3[-1] == 448.0 and len(E4M3) == 127


def nearest(v: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """The grid value (grid[code], codes in order of magnitude) nearest to |v| with v's sign; a
    tie goes to the even code; values past the largest saturate."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return np.copysign(grid[pick], v)


def scale_of(amax: np.ndarray, fmt: str) -> np.ndarray:
    """Scale per block from its largest magnitude, in 64 bits."""
    top = TOP[fmt]
    with np.errstate(divide="ignore"):
        if fmt == "blockwise":
            s = np.maximum(amax / top, 2.0 ** -126)
        elif fmt == "nvfp4":
            s = nearest(np.maximum(amax / top, 2.0 ** -9), E4M3)
        else:
            m, e = np.frexp(amax / top)  # m in [0.5, 1): 2^(e-1) exactly where m == 0.5
            s = np.ldexp(1.0, np.clip(np.where(m == 0.5, e - 1, e), -127, 127))
    return np.where(amax == 0, 1.0, s)


def decode(q: torch.Tensor, scales: torch.Tensor, fmt: str, rows: int, K: int):
    """(values of the codes [rows, K], scales [rows, K/vec]) as numpy float64."""
    q = q.reshape(rows, -1).cpu()
    if fmt in ("mxfp4", "nvfp4"):
        b = q.numpy()
        code = np.stack([b & 15, b >> 4], axis=-1).reshape(rows, K)
        v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    else:
        v = q.view(torch.float8_e4m3fn).double().numpy()
    s = scales.cpu()
    if fmt == "blockwise":
        s = s.reshape(K // 128, rows).t().double().numpy()
    elif fmt == "nvfp4":
        s = s.reshape(rows, -1).view(torch.float8_e4m3fn).double().numpy()
    else:
        s = s.reshape(rows, -1).view(torch.float8_e8m0fnu).double().numpy()
    return v, np.ascontiguousarray(s)


def check_quantised(v: np.ndarray, q: torch.Tensor, scales: torch.Tensor, fmt: str,
                    u_value, u_scale: float) -> None:
    """v [rows, K]: exact values; u_value: relative error of what is rounded (number or array);
    u_scale: of the block's largest magnitude and of the scale's own arithmetic."""
    rows, K = v.shape
    vec, grid = VEC[fmt], E2M1 if "fp4" in fmt else E4M3
    got, s = decode(q, scales, fmt, rows, K)
    a = np.abs(v).reshape(rows, K // vec, vec).max(-1)
    ua = np.broadcast_to(np.asarray(u_value, np.float64), v.shape).reshape(rows, K // vec, vec).max(-1)
    lo, hi = scale_of(a * (1 - ua - u_scale), fmt), scale_of(a * (1 + ua + u_scale), fmt)
    lo, hi = np.where(a == 0, 1.0, lo), np.where(a == 0, 1.0, hi)
    if fmt == "blockwise":
        lo, hi = lo * (1 - u_scale), hi * (1 + u_scale)
    bad = ~((s >= lo) & (s <= hi))
    assert not bad.any(), (fmt, "scales", int(bad.sum()), s[bad][:4], lo[bad][:4], hi[bad][:4])
    x = v / np.repeat(s, vec, axis=1)
    one, two = nearest(x * (1 - u_value), grid), nearest(x * (1 + u_value), grid)
    bad = ~((got == one) | (got == two) | (np.minimum(one, two) <= got) & (got <= np.maximum(one, two)))
    assert not bad.any(), (fmt, "codes", int(bad.sum()), got[bad][:4], x[bad][:4])


def sort_slots(ids: np.ndarray, experts: int):
    """(offsets [E+2], row_of_slot, slot_of_row) of flat ids."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(experts + 2)).astype(np.int32)
    row = np.empty(len(flat), np.int32)
    row[order] = np.arange(len(flat))
    slot = order.astype(np.int32)
    row[key == experts] = -1
    slot[offsets[experts]:] = -1
    return offsets, row, slot


def combine(C, row, weights, residual):
    """(sum [T, N], sum of magnitudes [T, N]) in float64; row [T, k], C [rows, N]."""
    T, k = row.shape
    out = np.zeros((T, C.shape[1])) if residual is None else residual.copy()
    mag = np.abs(out)
    for j in range(k):
        live = row[:, j] >= 0
        w = 1.0 if weights is None else weights[live, j][:, None]
        term = w * C[row[live, j]]
        out[live] += term
        mag[live] += np.abs(term)
    return out, mag


def combine_backward(d_out, C, row, weights):
    """(dC of the named rows by row, d_weights, sum of magnitudes per weight) in float64."""
    T, k = row.shape
    dC = np.full_like(C, np.nan)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        live = np.nonzero(row[:, j] >= 0)[0]
        r = row[live, j]
        dC[r] = weights[live, j][:, None] * d_out[live]
        p = d_out[live] * C[r]
        dw[live, j], mag[live, j] = p.sum(1), np.abs(p).sum(1)
    return dC, dw, mag
