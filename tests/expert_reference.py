"""The experts' products, their gradients and SwiGLU's gradient in 64 bits, written from their
definitions on the CPU (torch float64), with the sums of magnitudes that the tolerances go by."""
from __future__ import annotations

import torch

E4M3 = torch.float8_e4m3fn
BLOCK = 128
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# the smallest step of a type, halved: what a rounding may cost where the value is subnormal
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def offsets_of(sizes):
    return torch.tensor([0] + list(sizes)).cumsum(0).to(torch.int32)


def product(A, B, offsets, ids, transposed: bool):
    """(C [rows, N], sum of magnitudes) of the rows up to the last group's end."""
    off = offsets.tolist()
    N = B.shape[2] if transposed else B.shape[1]
    C, T = torch.zeros(off[-1], N, dtype=torch.float64), torch.zeros(off[-1], N, dtype=torch.float64)
    for g, (r0, r1) in enumerate(zip(off, off[1:])):
        if r1 > r0:
            W = B[g if ids is None else int(ids[g])].double()
            W = W if transposed else W.t()
            C[r0:r1] = A[r0:r1].double() @ W
            T[r0:r1] = A[r0:r1].double().abs() @ W.abs()
    return C, T


def wgrad(dC, A, offsets):
    """(dB [experts, N, K], sum of magnitudes) of values."""
    off = offsets.tolist()
    shape = (len(off) - 1, dC.shape[1], A.shape[1])
    dB, T = torch.zeros(shape, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
    for e, (r0, r1) in enumerate(zip(off, off[1:])):
        x, y = dC[r0:r1].double(), A[r0:r1].double()
        dB[e], T[e] = x.t() @ y, x.abs().t() @ y.abs()
    return dB, T


def blocks_of(offsets):
    """[(row of the scales, first row, end)] of every block of 128 rows."""
    off = offsets.tolist()
    return [(r0 // BLOCK + e + j, r, min(r + BLOCK, r1)) for e, (r0, r1) in enumerate(zip(off, off[1:]))
            for j, r in enumerate(range(r0, r1, BLOCK))]


def dequantised_columns(codes, scales, offsets):
    """Values of e4m3 codes [rows, K] with a scale for each block of 128 rows of a column."""
    out = torch.zeros(codes.shape, dtype=torch.float64)
    for s, r0, r1 in blocks_of(offsets):
        out[r0:r1] = codes[r0:r1].view(E4M3).double() * scales[s].double()
    return out


def quantise_columns(x, offsets):
    """(codes uint8, scales) as bsfp8_quantize_columns defines them, for inputs of other tests."""
    rows, K = x.shape
    q = torch.zeros(rows, K, dtype=torch.uint8)
    scales = torch.zeros(rows // BLOCK + offsets.numel() - 1, K)
    for s, r0, r1 in blocks_of(offsets):
        a = x[r0:r1].double().abs().amax(0)
        scales[s] = torch.where(a == 0, 1.0, a / 448).float()
        q[r0:r1] = (x[r0:r1].double() / scales[s].double()).clamp(-448, 448).float().to(E4M3).view(torch.uint8)
    return q, scales


def swiglu_backward(h, d_act):
    """(act, d_h, magnitude of what d_h's terms are, per element) in float64."""
    g, u = h.double().chunk(2, dim=1)
    d = d_act.double()
    s = torch.special.expit(g)
    r = torch.special.expit(-g)
    act = g * s * u
    d_h = torch.cat([d * u * s * (1 + g * r), d * g * s], dim=1)
    mag = torch.cat([(d * u * s).abs() * (1 + g.abs() * r), (d * g * s).abs()], dim=1)
    return act, d_h, mag
