"""A mixture-of-experts layer on the framework's operators, from the residual stream to the
residual stream, for any operand format:

    layer = MoeLayer(norm_weight, router, gate_up, down, top_k=8, format="mxfp8", max_rows=4096)
    out, residual = layer(x, residual)

norm and residual -> router (torch) -> slots sorted by expert -> rows quantised into expert order
-> grouped GEMM -> SwiGLU, quantised -> grouped GEMM -> weighted sum per token.  Nothing is read
back to the host, so the call can be captured in a CUDA graph.

    python examples/moe_layer.py [--format mxfp8] [--rows 16] [--hidden 2048] [--ffn 1024]
                                 [--experts 16] [--top-k 4]

runs a layer with random weights, compares it with the same layer in fp32 and prints its time.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_persistent_gb300 as bsfp8

EPS = 1e-6


def operand(format: str, rows: int, K: int):
    """Buffers (q, scales) of an operand of rows x K."""
    q = torch.empty(rows, K // 2 if "fp4" in format else K, dtype=torch.uint8, device="cuda")
    if format == "blockwise":
        return q, torch.empty(K // 128, rows, device="cuda")
    return q, torch.empty(rows, K // (16 if format == "nvfp4" else 32), dtype=torch.uint8, device="cuda")


def quantised_weights(W: torch.Tensor, format: str):
    """Expert weights [E, N, K] as a grouped GEMM's B and its scales."""
    E, N, K = W.shape
    if format == "blockwise":  # 128 x 128 blocks
        blocks = W.float().reshape(E, N // 128, 128, K // 128, 128)
        scales = (blocks.abs().amax(dim=(2, 4)) / 448).clamp(min=2.0 ** -126)
        q = (blocks / scales[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        return q.reshape(E, N, K).view(torch.uint8), scales.contiguous()
    q, scales = operand(format, E * N, K)
    bsfp8.bsmx_quantize(format, W.reshape(E * N, K).contiguous(), q, scales, E * N, K)
    return q, scales


class MoeLayer:
    """gate_up [E, 2F, H] (gate rows, then up rows) and down [E, H, F] in bf16 or fp32, router
    [E, H].  Experts that `first_expert` and the number of experts here leave out belong to other
    ranks: their slots are dropped, and this rank's part of the sum comes back."""

    def __init__(self, norm_weight, router, gate_up, down, top_k: int, format: str, max_rows: int, first_expert: int = 0):
        self.E, two_f, self.H = gate_up.shape
        self.F, self.top_k, self.format, self.first = two_f // 2, top_k, format, first_expert
        self.norm_weight, self.router = norm_weight, router
        self.gate_up, self.down = quantised_weights(gate_up, format), quantised_weights(down, format)
        slots = max_rows * top_k
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.offsets, self.row_of_slot = i32(self.E + 2), i32(slots)
        self.workspace = torch.empty(max(4, bsfp8.bsmx_moe_sort_workspace(max_rows, top_k, self.E)), dtype=torch.uint8, device="cuda")
        # the rows of dropped slots are a last group under some expert; nothing reads its result
        self.group_expert = torch.arange(self.E + 1, dtype=torch.int32, device="cuda").clamp_(max=self.E - 1)

    def _product(self, A, B, C, rows: int, N: int, K: int):
        args = (A[0], B[0], A[1], B[1], self.offsets)
        if self.format == "blockwise":
            bsfp8.bsfp8_grouped_gemm_ids(*args, self.group_expert, C, rows, N, K, self.E + 1, self.E)
        else:
            bsfp8.bsmx_grouped_gemm(self.format, self.format, *args, C, rows, N, K, self.E + 1, self.E, expert_ids=self.group_expert)

    def route(self, y):
        """The router in torch: ids int32 [rows, top_k] of this rank's experts, weights fp32."""
        top, ids = torch.topk(y.float() @ self.router.float().t(), self.top_k, dim=1)
        return (ids - self.first).to(torch.int32), torch.softmax(top, dim=1)

    def __call__(self, x, residual, keep: dict | None = None):
        rows, H, F, fmt = x.shape[0], self.H, self.F, self.format
        slots = rows * self.top_k
        new = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        y, residual_out = new(rows, H), torch.empty_like(residual)
        bsfp8.bsmx_rmsnorm_quant(fmt, x, self.norm_weight, EPS, rows, H, residual=residual, residual_out=residual_out, y=y)
        ids, weights = self.route(y)
        bsfp8.bsmx_moe_sort(ids, self.offsets, self.row_of_slot, self.workspace, rows, self.top_k, self.E)
        A = operand(fmt, slots, H)
        bsfp8.bsmx_quantize(fmt, y, *A, rows, H, row_of_slot=self.row_of_slot, top_k=self.top_k, out_rows=slots)
        h = new(slots, 2 * F)
        self._product(A, self.gate_up, h, slots, 2 * F, H)
        A2 = operand(fmt, slots, F)
        bsfp8.bsmx_swiglu_quant(fmt, h, *A2, slots, F)
        C = new(slots, H)
        self._product(A2, self.down, C, slots, H, F)
        out = new(rows, H)
        bsfp8.bsmx_moe_combine(C, self.row_of_slot, out, rows, slots, self.top_k, H, weights=weights)
        if keep is not None:
            keep.update(y=y, ids=ids, weights=weights, A=A, h=h, A2=A2, C=C)
        return out, residual_out


def plain_layer(x, residual, norm_weight, router, gate_up, down, top_k: int):
    """The layer in fp32, expert by expert."""
    h = x.float() + residual.float()
    y = (h * torch.rsqrt(h.pow(2).mean(-1, keepdim=True) + EPS) * norm_weight.float()).to(torch.bfloat16).float()
    top, ids = torch.topk(y @ router.float().t(), top_k, dim=1)
    weights, out = torch.softmax(top, dim=1), torch.zeros_like(y)
    for e in range(gate_up.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        g, u = (y[t] @ gate_up[e].float().t()).chunk(2, dim=1)
        out.index_add_(0, t, weights[t, j, None] * ((torch.nn.functional.silu(g) * u) @ down[e].float().t()))
    return out, h


def random_layer(hidden: int, ffn: int, experts: int, seed: int = 0):
    """(norm weight, router, gate_up, down) of a layer with random bf16 weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda scale, *shape: (scale * torch.randn(*shape, device="cuda", generator=g)).to(torch.bfloat16)  # noqa: E731
    return ((1 + 0.1 * torch.randn(hidden, device="cuda", generator=g)).to(torch.bfloat16), r(hidden ** -0.5, experts, hidden),
            r(hidden ** -0.5, experts, 2 * ffn, hidden), r(ffn ** -0.5, experts, hidden, ffn))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--format", default="mxfp8", choices=sorted(bsfp8.QUANT_FORMATS))
    for name, value in (("rows", 16), ("hidden", 2048), ("ffn", 1024), ("experts", 16), ("top-k", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    weights = random_layer(a.hidden, a.ffn, a.experts)
    layer = MoeLayer(*weights, top_k=a.top_k, format=a.format, max_rows=a.rows)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual = (torch.randn(a.rows, a.hidden, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    out, _ = layer(x, residual)
    want, _ = plain_layer(x, residual, *weights, a.top_k)
    error = float((out.float() - want).norm() / want.norm())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, residual)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        graph.replay()
    begin.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if bsfp8.bsfp8_get_device_error() != 0:
        raise SystemExit("device error")
    print(f"{a.format}: {a.rows} tokens, hidden {a.hidden}, {a.experts} experts of {a.ffn}, top {a.top_k}: "
          f"{begin.elapsed_time(end) * 50:.1f} us a layer, {error:.3f} of the output's norm off fp32")


if __name__ == "__main__":
    main()
