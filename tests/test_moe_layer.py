"""The operators together, as examples/moe_layer.py runs them: every stage of a layer against the
64-bit definition of that stage on the values it was given, for every operand format, with all
experts here and with experts of other ranks dropped; and the layer in a CUDA graph."""
import os
import sys

import numpy as np
import pytest
import torch

import block_scaled_fp8_persistent_gb300 as bsfp8
import moe_reference as ref

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

H, F, E, TOP_K = 512, 256, 6, 3


def _layer(fmt, rows, dropped):
    import moe_layer
    weights = moe_layer.random_layer(H, F, E, seed=3)
    if fmt == "nvfp4":  # weights of a size that e4m3 scales hold well
        weights = weights[:2] + (weights[2] * 4, weights[3] * 4)
    norm, router, gate_up, down = weights
    here = slice(1, 4) if dropped else slice(0, E)
    layer = moe_layer.MoeLayer(norm, router, gate_up[here].contiguous(), down[here].contiguous(), TOP_K, fmt, max_rows=rows,
                               first_expert=here.start)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, r = (torch.randn(rows, H, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    return layer, x, r, weights


def _values(fmt, q, s, rows, K):
    v, sc = ref.decode(q, s, fmt, rows, K)
    return v * np.repeat(sc, ref.VEC[fmt], 1)


def _weights(fmt, q, s, E_, N, K):
    if fmt != "blockwise":
        return _values(fmt, q, s, E_ * N, K).reshape(E_, N, K)
    v = q.cpu().view(torch.float8_e4m3fn).double().numpy()
    return v * np.repeat(np.repeat(s.cpu().double().numpy(), 128, 1), 128, 2)


def _check_product(fmt, A, B, offsets, rows, kept, N, K, C, E_):
    a, b = _values(fmt, *A, rows, K), _weights(fmt, *B, E_, N, K)
    got = C.cpu().double().numpy()
    for e in range(E_):
        lo, hi = offsets[e], offsets[e + 1]
        want, mag = a[lo:hi] @ b[e].T, np.abs(a[lo:hi]) @ np.abs(b[e]).T
        ulp = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))) - 7)
        assert np.all(np.abs(got[lo:hi] - want) <= 2 * ulp + 1e-6 * mag)
    assert offsets[E_] == kept


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4", "blockwise"])
@pytest.mark.parametrize("rows", [1, 50, 900])
@pytest.mark.parametrize("dropped", [False, True])
def test_every_stage(fmt, rows, dropped):
    layer, x, r, _ = _layer(fmt, rows, dropped)
    keep = {}
    out, residual = layer(x, r, keep)
    assert bsfp8.bsfp8_get_device_error() == 0
    n, slots = layer.E, rows * TOP_K
    h = x.double().cpu() + r.double().cpu()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * layer.norm_weight.cpu().double()
    assert torch.all((keep["y"].cpu().double() - y).abs() <= y.abs() * (2.0 ** -8 + 2.0 ** -18))
    assert torch.equal(residual, (x.float() + r.float()).to(torch.bfloat16))
    offsets, row, slot = ref.sort_slots(keep["ids"].cpu().numpy(), n)
    assert np.array_equal(layer.offsets.cpu().numpy(), offsets)
    assert np.array_equal(layer.row_of_slot[:slots].cpu().numpy(), row)
    assert dropped == bool((row < 0).any()) or rows == 1
    kept = int(offsets[n])
    token = slot[:kept] // TOP_K
    u = {"mxfp8": (0.0, 0.0), "mxfp4": (0.0, 0.0), "nvfp4": (0.0, 2.0 ** -23), "blockwise": (2.0 ** -22, 2.0 ** -22)}[fmt]
    kept_of = lambda A: (A[0][:kept], A[1][:, :kept] if fmt == "blockwise" else A[1][:kept])  # noqa: E731
    if kept:
        ref.check_quantised(keep["y"].cpu().double().numpy()[token], *kept_of(keep["A"]), fmt, *u)
        _check_product(fmt, kept_of(keep["A"]), layer.gate_up, offsets, kept, kept, 2 * F, H, keep["h"][:kept], n)
        hv = keep["h"][:kept].cpu().double().numpy()
        gate, up = hv[:, :F], hv[:, F:]
        ref.check_quantised(gate / (1 + np.exp(-gate)) * up, *kept_of(keep["A2"]), fmt, (8 + np.abs(gate)) * 2.0 ** -22, 2.0 ** -21)
        _check_product(fmt, kept_of(keep["A2"]), layer.down, offsets, kept, kept, H, F, keep["C"][:kept], n)
    C = keep["C"].cpu().double().numpy()
    want, mag = ref.combine(C, row.reshape(rows, TOP_K), keep["weights"].cpu().double().numpy(), None)
    assert np.all(np.abs(out.cpu().double().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 5 * 2.0 ** -24 * mag)


@pytest.mark.parametrize("fmt,near", [("mxfp8", 0.1), ("blockwise", 0.1), ("mxfp4", 0.4), ("nvfp4", 0.3)])
def test_whole_layer_is_near_fp32(fmt, near):
    import moe_layer
    layer, x, r, weights = _layer(fmt, 128, False)
    out, _ = layer(x, r)
    want, _ = moe_layer.plain_layer(x, r, *weights, TOP_K)
    assert float((out.float() - want).norm() / want.norm()) < near


def test_layer_in_a_graph():
    layer, x, r, _ = _layer("mxfp8", 33, True)
    want = [t.clone() for t in layer(x, r)]
    first = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(x, r)
    x.normal_()  # other tokens, then the first ones again
    graph.replay()
    assert not torch.equal(got[0], want[0])
    x.copy_(first)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bsfp8.bsfp8_get_device_error() == 0


def test_example_runs(capsys, monkeypatch):
    import moe_layer
    monkeypatch.setattr(sys, "argv", ["moe_layer.py", "--rows", "5", "--hidden", "512", "--ffn", "256"])
    moe_layer.main()
    assert "us a layer" in capsys.readouterr().out
