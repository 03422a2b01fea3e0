"""The experts' operators together, as examples/moe_training.py runs them: every stage of a step
against the 64-bit definition of that stage on the values it was given, the step's gradients against
64-bit autograd and differences, and the step in a CUDA graph.

Tolerances of a stage are its operator's (test_expert_ops.py).  Those of a whole step are worst
cases, followed through the layer in 64 bits beside its values: a stage's result is off by the
derivative's magnitude times what its inputs are off, plus half a step of bf16 (2^-8 of it) where it
is rounded, plus (n / 16 + 2) 2^-23 of its terms' magnitudes for a sum of n.  That is to first order;
the inputs are off by less than 2^-3 of their terms' magnitude, and a quarter is added for the rest.
"""
import os
import sys

import numpy as np
import pytest
import torch

import block_scaled_fp8_persistent_gb300 as bsfp8
import expert_reference as ref
import moe_reference

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

H, F, E, TOP_K = 256, 128, 5, 3
BF16 = torch.bfloat16


def _step(fmt, rows, dropped, seed=0):
    """(the experts, their arguments): with dropped, ids go past the experts that are here."""
    import moe_training
    y, ids, weights, gate_up, down, d_out = moe_training.random_step(rows, H, F, E, TOP_K, seed, choices=2 * E if dropped else E)
    return moe_training.TrainedExperts(gate_up, down, TOP_K, fmt, max_rows=rows), (y, ids, weights), d_out


def _close(got, want, tol, dtype):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= tol + (want.abs() + tol) * ref.HALF[dtype] + ref.TINY[dtype])
    assert not bad.any(), (int(bad.sum()), bad.numel(), got[bad][:4].tolist(), want[bad][:4].tolist())


def _fp32(terms, n):
    return terms * (n / 16 + 2) * 2.0 ** -23


def _check_product(A, B, off, C, n, transposed):
    want, T = ref.product(A.cpu(), B.cpu(), off, None, transposed)
    _close(C[: want.shape[0]], want, _fp32(T, n), BF16)


def _values(q, s, rows, K):
    v, sc = moe_reference.decode(q, s, "blockwise", rows, K)
    return torch.from_numpy(v * np.repeat(sc, 128, 1))


def _weights(q, s):
    return q.cpu().view(ref.E4M3).double() * s.cpu().double().repeat_interleave(128, 1).repeat_interleave(128, 2)


def _check_blockwise(A, B, off, C, rows, K):
    a, kept = _values(*A, rows, K), int(off[-1])
    want, T = ref.product(a, _weights(*B), off, None, False)
    # the product's own tolerance in the block-scaled tests: two steps of bf16 and 1e-6 of the terms
    assert torch.all((C[:kept].double().cpu() - want).abs() <= want.abs() * 2.0 ** -6 + T * 1e-6)


def _check_columns(x, q, s, off):
    """q, s [..] are x quantised along the rows: each code within half a step."""
    kept = int(off[-1])
    x = x[:kept].double().cpu()
    v, step = ref.dequantised_columns(q.cpu(), s.cpu(), off)[:kept], torch.zeros_like(x)
    for row, r0, r1 in ref.blocks_of(off):
        a = x[r0:r1].abs().amax(0)
        assert torch.all((s[row].double().cpu() - torch.where(a == 0, torch.ones_like(a), a / 448)).abs() <= a * 2.0 ** -22 / 448)
        step[r0:r1] = s[row].double().cpu()
    assert torch.all((v - x).abs() <= (x.abs() * 2.0 ** -4).maximum(step * 2.0 ** -10) * (1 + 2.0 ** -17))


@pytest.mark.parametrize("fmt", ["bf16", "blockwise"])
@pytest.mark.parametrize("rows", [1, 50, 700])
@pytest.mark.parametrize("dropped", [False, True])
def test_every_stage(fmt, rows, dropped):
    experts, (y, ids, weights), d_out = _step(fmt, rows, dropped)
    start = [torch.randn_like(g) for g in (experts.d_gate_up, experts.d_down)]
    experts.d_gate_up.copy_(start[0])
    experts.d_down.copy_(start[1])
    out, kept = experts.forward(y, ids, weights)
    st = {}
    d_y, d_weights = experts.backward(d_out, kept, st)
    assert bsfp8.bsfp8_get_device_error() == 0
    slots = rows * TOP_K
    offsets, row, slot = moe_reference.sort_slots(ids.cpu().numpy(), E)
    off = torch.from_numpy(offsets[: E + 1].copy())
    n = int(off[-1])
    assert np.array_equal(kept["offsets"].cpu().numpy(), offsets)
    assert np.array_equal(kept["slot_of_row"].cpu().numpy()[:n], slot[:n])
    assert dropped == bool((row < 0).any())
    gathered = y.cpu()[torch.from_numpy(slot[:n].astype(np.int64)) // TOP_K]
    whole = torch.from_numpy(offsets)  # with the group of dropped rows
    if fmt == "bf16":
        _check_product(gathered, experts.gate_up, off, kept["h"], H, False)
        _check_product(kept["act"][:n], experts.down, off, kept["C"], F, False)
        _check_product(st["dC"][:n], experts.down, off, st["d_act"], H, True)
        _check_product(st["d_h"][:n], experts.gate_up, off, st["dA"], 2 * F, True)
        act, d_rows = kept["act"], None
    else:
        def requantised(x, K):
            import moe_layer
            q = moe_layer.operand("blockwise", slots, K)
            bsfp8.bsmx_quantize("blockwise", x, *q, slots, K)
            return q
        _check_blockwise(requantised(st["dC"], H), experts.qt["down"], off, st["d_act"], slots, H)
        _check_blockwise(st["d_rows"], experts.qt["gate_up"], off, st["dA"], slots, 2 * F)
        _check_columns(st["dC"], *st["dC_"], off)
        _check_columns(st["d_h"], *st["d_h_"], off)
        _check_columns(torch.cat([gathered, gathered.new_zeros(slots - n, H)]), *st["A"], off)
        act = None
    # SwiGLU and its gradient
    h, d_act = kept["h"][:n].cpu(), st["d_act"][:n].cpu()
    want_act, want, _ = ref.swiglu_backward(h, d_act)
    g, u, d = h[:, :F].double(), h[:, F:].double(), d_act.double()
    s = torch.special.expit(g)
    rounding = (10 + g.abs()) * 2.0 ** -22
    if act is not None:
        _close(act[:n], want_act, want_act.abs() * rounding, BF16)
    # (where g is near -1.28 the terms of the gate's gradient cancel: relative to them)
    terms = torch.cat([(d * u * s).abs() * (1 + g.abs()), (d * g * s).abs()], dim=1)
    _close(st["d_h"][:n], want, terms * torch.cat([rounding, rounding], dim=1), BF16)
    # the weights' gradients, added to what was there
    for name, dC, A, was in (("d_down", st["dC_"], st["act"], start[1]), ("d_gate_up", st["d_h_"], st["A"], start[0])):
        if fmt == "bf16":
            values = [x[:n].cpu() for x in (dC, A)]
        else:
            values = [ref.dequantised_columns(q.cpu(), sc.cpu(), off) for q, sc in (dC, A)]
        want, T = ref.wgrad(*values, off)
        was = was.double().cpu()
        tol = T * (max(np.diff(offsets[: E + 1])) / 16 + 6) * 2.0 ** -23 + (was.abs() + T) * 2.0 ** -24
        _close(getattr(experts, name), want + was, tol, torch.float32)
    # the sums per token and their gradient
    C, row = kept["C"].double().cpu().numpy(), row.reshape(rows, TOP_K)
    want, mag = moe_reference.combine(C, row, weights.double().cpu().numpy(), None)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 5 * 2.0 ** -24 * mag)
    want, mag = moe_reference.combine(st["dA"].double().cpu().numpy(), row, np.ones((rows, TOP_K)), None)
    assert np.all(np.abs(d_y.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 5 * 2.0 ** -24 * mag)
    assert torch.all(d_weights.cpu()[torch.from_numpy(row < 0)] == 0)


def _bounded_step(args, gate_up, down, d_out):
    """The step's gradients in float64 and how far a bf16 run of it may be off, by name."""
    y, ids, weights = (x.cpu() for x in args)
    W1, W2, d_out = gate_up.cpu().double(), down.cpu().double(), d_out.cpu().double()
    y, weights, half = y.double(), weights.double(), 2.0 ** -8
    rows = y.shape[0]
    v = dict(d_y=torch.zeros(rows, H), d_weights=torch.zeros(rows, TOP_K), d_gate_up=torch.zeros_like(W1), d_down=torch.zeros_like(W2))
    v = {k: x.double() for k, x in v.items()}
    e_ = {k: torch.zeros_like(x) for k, x in v.items()}

    def rounded(x, off):
        return off + half * (x.abs() + off)

    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        x, w = y[t], weights[t, j, None]
        h = x @ W1[e].t()
        eh = rounded(h, _fp32(x.abs() @ W1[e].abs().t(), H))
        g, u = h.chunk(2, dim=1)
        eg, eu = eh.chunk(2, dim=1)
        s = torch.special.expit(g)
        phi, phi1, phi2 = g * s, s * (1 + g * (1 - s)), s * (1 - s) * (2 + g * (1 - 2 * s))
        act = phi * u
        ea = rounded(act, (phi1 * u).abs() * eg + phi.abs() * eu + (10 + g.abs()) * 2.0 ** -22 * act.abs())
        C = act @ W2[e].t()
        eC = rounded(C, ea @ W2[e].abs().t() + _fp32(act.abs() @ W2[e].abs().t(), F))
        dC = w * d_out[t]
        edC = rounded(dC, dC.abs() * 2.0 ** -24)
        v["d_weights"][t, j] = (d_out[t] * C).sum(1)
        e_["d_weights"][t, j] = (d_out[t].abs() * eC).sum(1) + H * 2.0 ** -24 * (d_out[t] * C).abs().sum(1)
        d = dC @ W2[e]
        ed = rounded(d, edC @ W2[e].abs() + _fp32(dC.abs() @ W2[e].abs(), H))
        v["d_down"][e] = dC.t() @ act
        e_["d_down"][e] = edC.t() @ act.abs() + dC.abs().t() @ ea + _fp32(dC.abs().t() @ act.abs(), t.numel())
        d_h = torch.cat([d * u * phi1, d * phi], dim=1)
        terms = torch.cat([(d * u * s).abs() * (1 + g.abs()), (d * phi).abs()], dim=1) * (10 + g.abs()).repeat(1, 2) * 2.0 ** -22
        ed_h = torch.cat([(u * phi1).abs() * ed + (d * phi1).abs() * eu + (d * u * phi2).abs() * eg,
                          phi.abs() * ed + (d * phi1).abs() * eg], dim=1)
        ed_h = rounded(d_h, ed_h + terms)
        v["d_gate_up"][e] = d_h.t() @ x
        e_["d_gate_up"][e] = ed_h.t() @ x.abs() + _fp32(d_h.abs().t() @ x.abs(), t.numel())
        dA = d_h @ W1[e]
        edA = rounded(dA, ed_h @ W1[e].abs() + _fp32(d_h.abs() @ W1[e].abs(), 2 * F))
        v["d_y"].index_add_(0, t, dA)
        e_["d_y"].index_add_(0, t, edA)
    e_["d_y"] = rounded(v["d_y"], e_["d_y"] * (1 + 2.0 ** -20))
    return v, {k: x * 1.25 for k, x in e_.items()}


@pytest.mark.parametrize("rows,dropped", [(3, False), (64, True), (400, False)])
def test_gradients(rows, dropped):
    """Against 64-bit autograd of the plain layer, and along their own direction against differences
    of the layer's 64-bit loss."""
    import moe_training
    experts, args, d_out = _step("bf16", rows, dropped, seed=rows)
    out, kept = experts.forward(*args)
    d_y, d_weights = experts.backward(d_out, kept)
    got = dict(d_y=d_y, d_weights=d_weights, d_gate_up=experts.d_gate_up, d_down=experts.d_down)
    got = {k: x.double().cpu() for k, x in got.items()}
    want, off = _bounded_step(args, experts.gate_up, experts.down, d_out)
    names = ("d_y", "d_weights", "d_gate_up", "d_down")
    y, ids, weights = (x.cpu() for x in args)
    leaves = [x.double().cpu().requires_grad_() for x in (y, weights, experts.gate_up, experts.down)]
    loss = lambda *p: (moe_training.plain_experts(p[0], ids, *p[1:]) * d_out.double().cpu()).sum()  # noqa: E731
    for name, grad in zip(names, torch.autograd.grad(loss(*leaves), leaves)):
        assert torch.allclose(want[name], grad, rtol=1e-9, atol=1e-9 * float(grad.abs().max()))
        assert torch.all((got[name] - grad).abs() <= off[name]), name
    with torch.no_grad():
        for i, name in enumerate(names):
            v = got[name] / got[name].norm()
            at = lambda step: loss(*[x + step * v if k == i else x for k, x in enumerate(leaves)])  # noqa: E731,B023
            slope = float((at(1e-4) - at(-1e-4)) / 2e-4)
            # (a central difference is off by step^2 / 6 of the third derivative along v)
            assert abs(float((got[name] * v).sum()) - slope) <= float((off[name] * v.abs()).sum()) + 1e-5 * abs(slope)


@pytest.mark.parametrize("fmt", ["bf16", "blockwise"])
def test_nothing_kept(fmt):
    """Every slot dropped: no gradients, and what was added up stays."""
    experts, (y, ids, weights), d_out = _step(fmt, 9, False)
    experts.d_gate_up.fill_(2.5)
    out, kept = experts.forward(y, torch.full_like(ids, -1), weights)
    d_y, d_weights = experts.backward(d_out, kept)
    assert bsfp8.bsfp8_get_device_error() == 0
    for x in (out, d_y, d_weights, experts.d_down, experts.d_gate_up - 2.5):
        assert torch.all(x == 0)


@pytest.mark.parametrize("fmt", ["bf16", "blockwise"])
def test_step_in_a_graph(fmt):
    experts, args, d_out = _step(fmt, 77, True)

    def step():
        experts.d_gate_up.zero_()
        experts.d_down.zero_()
        out, kept = experts.forward(*args)
        return (out, *experts.backward(d_out, kept), experts.d_gate_up, experts.d_down)

    want = [x.clone() for x in step()]
    first = [x.clone() for x in (*args, d_out)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    args[0].normal_()  # other tokens, other choices, then the first ones again
    args[1].copy_(args[1].flip(0))
    d_out.normal_()
    graph.replay()
    assert not any(torch.equal(a, b) for a, b in zip(got, want))
    for x, was in zip((*args, d_out), first):
        x.copy_(was)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bsfp8.bsfp8_get_device_error() == 0


@pytest.mark.parametrize("fmt", ["bf16", "blockwise"])
def test_example_runs(fmt, capsys, monkeypatch):
    import moe_training
    monkeypatch.setattr(sys, "argv", ["moe_training.py", "--format", fmt, "--rows", "60", "--hidden", "256", "--ffn", "128"])
    moe_training.main()
    assert "forward and backward" in capsys.readouterr().out
