"""The experts of a mixture-of-experts layer trained on the framework's operators, forward and
backward, in bf16 or with every product in block-scaled FP8:

    experts = TrainedExperts(gate_up, down, top_k=8, format="bf16", max_rows=4096)
    out, kept = experts.forward(y, ids, weights)
    d_y, d_weights = experts.backward(d_out, kept)      # adds to d_gate_up and d_down (fp32)

forward:  slots sorted by expert -> rows in expert order -> grouped product -> SwiGLU -> grouped
product -> weighted sum per token.  backward: the sum's gradient, then for each of the two products
its rows' gradient and its weights', with SwiGLU's between them.  In FP8 an operand is quantised
along its columns for the products and along its rows for the weights' gradients.  Nothing is read
back to the host, so both can be captured in a CUDA graph.

    python examples/moe_training.py [--format bf16|blockwise] [--rows 4096] [--hidden 2048]
                                    [--ffn 1024] [--experts 16] [--top-k 4]

takes a step with random weights, compares the gradients with the same layer's in fp32 and prints
its time.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import block_scaled_fp8_persistent_gb300 as bsfp8
if __package__:
    from .moe_layer import operand, quantised_weights
else:
    from moe_layer import operand, quantised_weights


class TrainedExperts:
    """gate_up [E, 2F, H] (gate rows, then up rows) and down [E, H, F] in bf16; their gradients are
    d_gate_up and d_down in fp32, added to by every backward().  Slots whose id is outside [0, E)
    are dropped."""

    def __init__(self, gate_up, down, top_k: int, format: str, max_rows: int):
        if format not in ("bf16", "blockwise"):
            raise ValueError("format: bf16 or blockwise")
        self.E, two_f, self.H = gate_up.shape
        self.F, self.top_k, self.format = two_f // 2, top_k, format
        self.gate_up, self.down = gate_up, down
        self.d_gate_up, self.d_down = (torch.zeros_like(w, dtype=torch.float32) for w in (gate_up, down))
        if format == "blockwise":
            self.refresh()
        self.workspace = torch.empty(max(4, bsfp8.bsmx_moe_sort_workspace(max_rows, top_k, self.E)), dtype=torch.uint8, device="cuda")
        # a block-scaled product takes whole batches: the rows of dropped slots are a last group
        # under some expert, and nothing reads its result
        self.group_expert = torch.arange(self.E + 1, dtype=torch.int32, device="cuda").clamp_(max=self.E - 1)

    def refresh(self):
        """Quantises the weights, as they lie and transposed (after every optimizer step)."""
        self.q = {w: quantised_weights(getattr(self, w), "blockwise") for w in ("gate_up", "down")}
        # blocks of 128 x 128: the transpose has the same codes and scales
        self.qt = {w: tuple(x.transpose(1, 2).contiguous() for x in self.q[w]) for w in self.q}

    def _product(self, kept, A, weight: str, rows: int, N: int, K: int, transposed: bool):
        C = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        if self.format == "bf16":
            bsfp8.bs16_grouped_gemm(A, getattr(self, weight), kept["offsets"], C, rows, N, K, self.E, self.E, transposed=transposed)
        else:
            q, scales = (self.qt if transposed else self.q)[weight]
            bsfp8.bsfp8_grouped_gemm_ids(A[0], q, A[1], scales, kept["offsets"], self.group_expert, C, rows, N, K, self.E + 1, self.E)
        return C

    def _columns(self, kept, x, rows: int, K: int, gathered: bool = False):
        q = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
        scales = torch.empty(rows // 128 + self.E, K, device="cuda")
        by = dict(slot_of_row=kept["slot_of_row"], top_k=self.top_k) if gathered else {}
        bsfp8.bsfp8_quantize_columns(x, kept["offsets"], q, scales, rows, K, self.E, **by)
        return q, scales

    def _wgrad(self, kept, dC, A, dB, rows: int, N: int, K: int):
        if self.format == "bf16":
            bsfp8.bs16_grouped_wgrad(dC, A, kept["offsets"], dB, rows, N, K, self.E, add=dB)
        else:
            bsfp8.bsfp8_grouped_wgrad(dC[0], A[0], dC[1], A[1], kept["offsets"], dB, rows, N, K, self.E, add=dB)

    def forward(self, y, ids, weights):
        """y bf16 [rows, H], ids int32 and weights fp32 [rows, top_k]: (out, what backward needs)."""
        rows, H, F, k = y.shape[0], self.H, self.F, self.top_k
        slots = rows * k
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        kept = dict(y=y, weights=weights, offsets=i32(self.E + 2), row_of_slot=i32(slots), slot_of_row=i32(slots))
        bsfp8.bsmx_moe_sort(ids, kept["offsets"], kept["row_of_slot"], self.workspace, rows, k, self.E, slot_of_row=kept["slot_of_row"])
        act = torch.empty(slots, F, dtype=torch.bfloat16, device="cuda")
        if self.format == "bf16":
            A = kept["A"] = y[kept["slot_of_row"].clamp(min=0) // k]
            h = self._product(kept, A, "gate_up", slots, 2 * F, H, False)
            bsfp8.bsmx_swiglu_backward(h, None, slots, F, act=act)
            C = self._product(kept, act, "down", slots, H, F, False)
            kept["act"] = act
        else:
            A, A2 = operand("blockwise", slots, H), operand("blockwise", slots, F)
            bsfp8.bsmx_quantize("blockwise", y, *A, rows, H, row_of_slot=kept["row_of_slot"], top_k=k, out_rows=slots)
            h = self._product(kept, A, "gate_up", slots, 2 * F, H, False)
            bsfp8.bsmx_swiglu_quant("blockwise", h, *A2, slots, F)
            C = self._product(kept, A2, "down", slots, H, F, False)
        out = torch.empty_like(y)
        bsfp8.bsmx_moe_combine(C, kept["row_of_slot"], out, rows, slots, k, H, weights=weights)
        kept.update(h=h, C=C)
        return out, kept

    def backward(self, d_out, kept, stages: dict | None = None):
        """(d_y bf16, d_weights fp32) of d_out bf16 [rows, H]."""
        rows, H, F, k = d_out.shape[0], self.H, self.F, self.top_k
        slots = rows * k
        new = lambda n: torch.empty(slots, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        dC, d_weights = new(H), torch.empty_like(kept["weights"])
        bsfp8.bsmx_moe_combine_backward(d_out, kept["C"], kept["row_of_slot"], kept["weights"], dC, d_weights, rows, slots, k, H)
        d_h = new(2 * F)
        if self.format == "bf16":
            d_act = self._product(kept, dC, "down", slots, F, H, True)
            dC_, act, d_h_, A = dC, kept["act"], d_h, kept["A"]
            bsfp8.bsmx_swiglu_backward(kept["h"], d_act, slots, F, d_h=d_h)
            d_rows = d_h
        else:
            q = operand("blockwise", slots, H)
            bsfp8.bsmx_quantize("blockwise", dC, *q, slots, H)
            d_act = self._product(kept, q, "down", slots, F, H, True)
            act16, d_rows = new(F), operand("blockwise", slots, 2 * F)
            bsfp8.bsmx_swiglu_backward(kept["h"], d_act, slots, F, d_h=d_h, act=act16, q=d_rows[0], scales=d_rows[1])
            dC_, act, d_h_ = (self._columns(kept, x, slots, n) for x, n in ((dC, H), (act16, F), (d_h, 2 * F)))
            A = self._columns(kept, kept["y"], slots, H, gathered=True)
        self._wgrad(kept, dC_, act, self.d_down, slots, H, F)
        self._wgrad(kept, d_h_, A, self.d_gate_up, slots, 2 * F, H)
        dA = self._product(kept, d_rows, "gate_up", slots, H, 2 * F, True)
        d_y = torch.empty_like(d_out)
        bsfp8.bsmx_moe_combine(dA, kept["row_of_slot"], d_y, rows, slots, k, H)
        if stages is not None:
            stages.update(dC=dC, dC_=dC_, d_act=d_act, act=act, d_h=d_h, d_h_=d_h_, d_rows=d_rows, A=A, dA=dA)
        return d_y, d_weights


def plain_experts(y, ids, weights, gate_up, down):
    """The experts in the arguments' type, expert by expert, for autograd."""
    out = torch.zeros_like(y)
    for e in range(gate_up.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        g, u = (y[t] @ gate_up[e].t()).chunk(2, dim=1)
        out = out.index_add(0, t, weights[t, j, None] * ((torch.nn.functional.silu(g) * u) @ down[e].t()))
    return out


def random_step(rows: int, hidden: int, ffn: int, experts: int, top_k: int, seed: int = 0, choices: int | None = None):
    """(y, ids, weights, gate_up, down, d_out) of random values; ids from 0 to choices - 1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda scale, *shape: (scale * torch.randn(*shape, device="cuda", generator=g)).to(torch.bfloat16)  # noqa: E731
    scores = torch.rand(rows, choices or experts, device="cuda", generator=g)
    top, ids = torch.topk(scores, top_k, dim=1)
    return (r(1.0, rows, hidden), ids.to(torch.int32), torch.softmax(top, dim=1), r(hidden ** -0.5, experts, 2 * ffn, hidden),
            r(ffn ** -0.5, experts, hidden, ffn), r(1.0, rows, hidden))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--format", default="bf16", choices=["bf16", "blockwise"])
    for name, value in (("rows", 4096), ("hidden", 2048), ("ffn", 1024), ("experts", 16), ("top-k", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    y, ids, weights, gate_up, down, d_out = random_step(a.rows, a.hidden, a.ffn, a.experts, a.top_k)
    experts = TrainedExperts(gate_up, down, a.top_k, a.format, max_rows=a.rows)

    def step():
        out, kept = experts.forward(y, ids, weights)
        return (out, *experts.backward(d_out, kept))

    out, d_y, d_weights = step()
    plain = [x.float().requires_grad_() for x in (y, weights, gate_up, down)]
    want = plain_experts(plain[0], ids, *plain[1:])
    grads = torch.autograd.grad(want, plain, d_out.float())
    pairs = zip(("out", "d_y", "d_weights", "d_gate_up", "d_down"), (out, d_y, d_weights, experts.d_gate_up, experts.d_down),
                (want, *grads))
    errors = ", ".join(f"{n} {float((x.float() - w.detach()).norm() / w.detach().norm()):.4f}" for n, x, w in pairs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
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
          f"{begin.elapsed_time(end) * 50:.1f} us forward and backward; of the norm off fp32: {errors}")


if __name__ == "__main__":
    main()
