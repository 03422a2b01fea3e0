"""The experts' products in 16 bits and the backward pass of the experts, as measured cases.

Each case is one pass through one operator of

    h = x W1ᵀ  ->  act = silu(gate) * up  ->  y = act W2ᵀ          (rows grouped by expert)

and of its gradients: the product in 16 bits, its input gradient (the weights read as they lie), its
weight gradient in 16 bits and in 8 bits with a scale for each 128 rows of a column, the operands of
the latter (rows quantised along the columns), and the activation's gradient; in its plain form
(elementary torch operations in fp32, each output rounded once) or, with `own` set, through the
framework's entry points.  e4m3 codes come back as float8 values beside their scales.
"""
import math

import torch

own = False

SEED_MIX = 1_000_003
E4M3 = torch.float8_e4m3fn
BLOCK = 128  # rows that share a scale
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of a small layer, two experts: latency of a call
        {"name": "product one token", "op": "product", "rows": 2, "N": 1024, "K": 2048, "experts": 8, "type": "bf16", "transposed": False},
        # a decode batch over 128 experts, a few rows each: the weights' bytes
        {"name": "product decode", "op": "product", "rows": 2091, "N": 4096, "K": 2048, "experts": 128, "type": "bf16", "transposed": False},
        # a prefill batch of 8 experts
        {"name": "product prefill", "op": "product", "rows": 4096, "N": 4096, "K": 7168, "experts": 8, "type": "bf16", "transposed": False},
        # gradient of a training batch's rows, 64 experts: the weights are read the other way round
        {"name": "input gradient", "op": "product", "rows": 16384, "N": 7168, "K": 2048, "experts": 64, "type": "fp16", "transposed": True},
        # weight gradient of a short fine-tuning sequence, in the weights' own type
        {"name": "weight gradient short", "op": "wgrad", "rows": 154, "N": 2048, "K": 1024, "experts": 8, "type": "bf16", "out": "bf16", "add": False, "dropped": 0.0},
        # of a training batch, added to fp32 gradients; a tenth of the rows belongs to no expert here
        {"name": "weight gradient", "op": "wgrad", "rows": 16384, "N": 2048, "K": 7168, "experts": 64, "type": "bf16", "out": "fp32", "add": True, "dropped": 0.1},
        # the same in 8 bits: a short sequence, and a long batch over 8 experts
        {"name": "fp8 weight gradient short", "op": "wgrad8", "rows": 301, "N": 2048, "K": 1024, "experts": 8, "out": "fp32", "add": False, "dropped": 0.0},
        {"name": "fp8 weight gradient", "op": "wgrad8", "rows": 16384, "N": 4096, "K": 7168, "experts": 8, "out": "fp32", "add": False, "dropped": 0.0},
        # operands of that gradient: a short sequence's gradient rows, and a batch's tokens gathered by expert
        {"name": "columns short", "op": "columns", "rows": 301, "K": 2048, "experts": 8, "top_k": 0, "dropped": 0.0},
        {"name": "columns gathered", "op": "columns", "rows": 8192, "K": 7168, "experts": 64, "top_k": 8, "dropped": 0.1},
        # the activation's gradient: of a short sequence in 16 bits, and of a batch as the next products' operands
        {"name": "swiglu gradient short", "op": "swiglu_grad", "rows": 154, "N": 1024, "type": "bf16", "act": False, "quantised": False},
        {"name": "swiglu gradient", "op": "swiglu_grad", "rows": 65536, "N": 2048, "type": "bf16", "act": True, "quantised": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, step):
    return step * _log_int(rng, lo // step, hi // step)


def draw(rng):
    op = rng.choice(["product", "product", "wgrad", "wgrad8", "columns", "swiglu_grad"])
    experts = rng.choice([1, 3, 8, 16, 60, 64, 128])
    if op == "product":
        return {"op": op, "rows": _log_int(rng, 1, 8192), "N": _width(rng, 128, 4096, 8), "K": _width(rng, 128, 4096, 8), "experts": experts,
                "type": rng.choice(["bf16", "fp16"]), "transposed": rng.random() < 0.5}
    if op == "wgrad":
        return {"op": op, "rows": _log_int(rng, 1, 8192), "N": _width(rng, 128, 2048, 8), "K": _width(rng, 128, 2048, 8), "experts": experts,
                "type": rng.choice(["bf16", "fp16"]), "out": rng.choice(["own", "fp32"]), "add": rng.random() < 0.5, "dropped": rng.choice([0.0, 0.1])}
    if op == "wgrad8":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "N": _width(rng, 128, 2048, 128), "K": _width(rng, 128, 2048, 128), "experts": experts,
                "out": rng.choice(["bf16", "fp32"]), "add": rng.random() < 0.5, "dropped": rng.choice([0.0, 0.1])}
    if op == "columns":
        return {"op": op, "rows": _log_int(rng, 1, 8192), "K": _width(rng, 128, 7168, 128), "experts": experts, "top_k": rng.choice([0, 1, 2, 8]),
                "dropped": rng.choice([0.0, 0.1])}
    return {"op": op, "rows": _log_int(rng, 1, 32768), "N": _width(rng, 128, 4096, 128), "type": rng.choice(["bf16", "fp16"]),
            "act": rng.random() < 0.5, "quantised": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * SEED_MIX % (1 << 62))
    return g


def _activations(g, rows, K, dtype=torch.bfloat16, spread=1.0):
    """Rows of normal values whose size differs from row to row, some channels being outliers."""
    size = torch.exp(0.5 * torch.randn(rows, 1, device="cuda", generator=g))
    channel = 1.0 + 15.0 * (torch.rand(K, device="cuda", generator=g) < 0.005)
    return torch.randn(rows, K, device="cuda", generator=g).mul_(size).mul_(channel).mul_(spread).to(dtype)


def _groups(g, rows, experts, dropped):
    """(offsets int32 [experts + 1], longest group) of rows that choose experts of uneven
    popularity; of three experts or more one gets none, and a share `dropped` of the rows lies
    behind the last group."""
    kept = rows - int(rows * dropped)
    p = torch.exp(0.4 * torch.randn(experts, device="cuda", generator=g))
    if experts > 2:
        p[experts // 2] = 0.0
    sizes = torch.bincount(torch.multinomial(p, kept, replacement=True, generator=g), minlength=experts)
    offsets = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).to(torch.int32)
    return offsets, int(sizes.max())


def _scale_row(offsets, rows):
    """Of every row: its group (experts for a row behind the last), and the row of the scales that
    its block of 128 rows has: blocks are counted from each group's first row, and block j of
    group e has row offsets[e] / 128 + e + j."""
    off = offsets.long()
    r = torch.arange(rows, device=off.device)
    group = torch.searchsorted(off[1:].contiguous(), r, right=True)
    first = off[group]
    return group, first // BLOCK + group + (r - first) // BLOCK


def _quantised_columns(x, offsets):
    """(e4m3 codes [rows, K], fp32 scales [rows / 128 + groups, K]) of fp32 rows; zeros for what
    belongs to no group."""
    rows, K = x.shape
    blocks = rows // BLOCK + offsets.numel() - 1
    group, at = _scale_row(offsets, rows)
    live = (group < offsets.numel() - 1)[:, None]
    at = torch.where(live[:, 0], at, 0)
    x = torch.where(live, x, 0.0)
    # every block's rows side by side; a row's place in its block is its distance from the group's first
    place = at * BLOCK + (torch.arange(rows, device=x.device) - offsets.long()[group]) % BLOCK
    place = torch.where(live[:, 0], place, blocks * BLOCK)
    side = torch.zeros(blocks * BLOCK + 1, K, device=x.device)
    side[place] = x
    amax = side[:-1].view(blocks, BLOCK, K).abs().amax(1)
    used = torch.zeros(blocks + 1, 1, dtype=torch.bool, device=x.device)
    used[torch.where(live[:, 0], at, blocks)] = True
    scale = torch.where(amax > 0, (amax / 448.0).clamp(min=2.0 ** -126), 1.0) * used[:-1]
    inverse = 1.0 / torch.where(scale > 0, scale, 1.0)
    return (x * inverse[at]).clamp(-448.0, 448.0).to(E4M3), scale


def prepare(case, seed):
    """Inputs, and the buffers that a program allocates once."""
    g, c = _gen(seed), dict(case)
    s = {"case": c}
    u8 = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    op, M = c["op"], c["rows"]
    if op == "product":
        dtype = TYPES[c["type"]]
        s["offsets"], s["longest"] = _groups(g, M, c["experts"], 0.0)
        s["A"] = _activations(g, M, c["K"], dtype)
        shape = (c["experts"], c["K"], c["N"]) if c["transposed"] else (c["experts"], c["N"], c["K"])
        s["B"] = torch.randn(shape, device="cuda", dtype=dtype, generator=g).mul_(c["K"] ** -0.5)
        s["C"] = torch.zeros(M, c["N"], dtype=dtype, device="cuda")
    elif op in ("wgrad", "wgrad8"):
        E, N, K = c["experts"], c["N"], c["K"]
        s["offsets"], s["longest"] = _groups(g, M, E, c["dropped"])
        dtype = TYPES[c["type"]] if op == "wgrad" else torch.float32
        s["dC"] = _activations(g, M, N, dtype, 0.01)
        s["A"] = _activations(g, M, K, dtype)
        if op == "wgrad8":
            codes, s["dc_scales"] = _quantised_columns(s["dC"], s["offsets"])
            s["dC"] = codes.view(torch.uint8)
            codes, s["a_scales"] = _quantised_columns(s["A"], s["offsets"])
            s["A"] = codes.view(torch.uint8)
        out = dtype if c["out"] == "own" else TYPES[c["out"]]
        s["dB"] = torch.zeros(E, N, K, dtype=out, device="cuda")
        s["add"] = torch.randn(E, N, K, device="cuda", dtype=out, generator=g).mul_(0.1) if c["add"] else None
    elif op == "columns":
        k, K, E = c["top_k"], c["K"], c["experts"]
        slots = M * max(k, 1)
        s["x"] = _activations(g, M, K)
        s["offsets"], _ = _groups(g, slots, E, c["dropped"])
        # the slot that lies in each row; those behind the last group hold none
        s["slot_of_row"] = None
        if k:
            slot = torch.randperm(slots, device="cuda", generator=g).to(torch.int32)
            slot[slots - int(slots * c["dropped"]):] = -1
            s["slot_of_row"] = slot
        s["q"], s["scales"] = u8(slots, K), torch.zeros(slots // BLOCK + E, K, device="cuda")
    else:
        dtype, N = TYPES[c["type"]], c["N"]
        s["h"] = _activations(g, M, 2 * N, dtype)
        s["d_act"] = _activations(g, M, N, dtype, 0.01)
        s["d_h"] = torch.zeros_like(s["h"])
        s["act"] = torch.zeros_like(s["d_act"]) if c["act"] else None
        s["q"], s["scales"] = (u8(M, 2 * N), torch.zeros(2 * N // BLOCK, M, device="cuda")) if c["quantised"] else (None, None)
    return s


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
def _side_by_side(x, offsets, longest):
    """Rows [rows, K] as fp32 [groups, longest, K], zeros behind each group's last row, and every
    row's (group, place); rows behind the last group are left out."""
    E = offsets.numel() - 1
    group, _ = _scale_row(offsets, x.shape[0])
    live = group < E
    place = torch.arange(x.shape[0], device=x.device) - offsets.long()[group]
    group, place = torch.where(live, group, E), torch.where(live, place, 0)
    out = torch.zeros(E + 1, max(longest, 1), x.shape[1], device=x.device)
    out[group, place] = torch.where(live[:, None], x.float(), 0.0)
    return out[:E], group, place


def _dequantised(codes, scales, offsets):
    group, at = _scale_row(offsets, codes.shape[0])
    at = torch.where(group < offsets.numel() - 1, at, 0)
    return codes.view(E4M3).float() * scales[at]


def _plain(s):
    c = s["case"]
    if c["op"] == "product":
        side, group, place = _side_by_side(s["A"], s["offsets"], s["longest"])
        B = s["B"].float()
        return torch.bmm(side, B if c["transposed"] else B.transpose(1, 2))[group, place].to(s["C"].dtype)
    if c["op"] in ("wgrad", "wgrad8"):
        dC, A = s["dC"], s["A"]
        if c["op"] == "wgrad8":
            dC, A = _dequantised(dC, s["dc_scales"], s["offsets"]), _dequantised(A, s["a_scales"], s["offsets"])
        dC, _, _ = _side_by_side(dC, s["offsets"], s["longest"])
        A, _, _ = _side_by_side(A, s["offsets"], s["longest"])
        dB = torch.bmm(dC.transpose(1, 2), A)
        if s["add"] is not None:
            dB += s["add"]
        return dB.to(s["dB"].dtype)
    if c["op"] == "columns":
        x = s["x"].float()
        if s["slot_of_row"] is not None:
            slot = s["slot_of_row"].long()
            x = x[slot.clamp(min=0) // c["top_k"]]
        q, scales = _quantised_columns(x, s["offsets"])
        return {"q": q, "scales": scales}
    gate, up, d = s["h"][:, : c["N"]].float(), s["h"][:, c["N"]:].float(), s["d_act"].float()
    sig = 1 / (1 + torch.exp(-gate))
    d_h = torch.cat([d * up * sig * (1 + gate * (1 - sig)), d * gate * sig], dim=1)
    out = {"d_h": d_h.to(s["h"].dtype)}
    if c["act"]:
        out["act"] = (gate * sig * up).to(s["h"].dtype)
    if c["quantised"]:
        b = d_h.view(c["rows"], -1, BLOCK)
        amax = b.abs().amax(-1)
        scale = torch.where(amax > 0, (amax / 448.0).clamp(min=2.0 ** -126), 1.0)
        out["q"] = (b * (1.0 / scale).unsqueeze(-1)).clamp(-448.0, 448.0).to(E4M3).view(c["rows"], -1)
        out["scales"] = scale.t().contiguous()
    return out


def _own(s):
    import block_scaled_fp8_persistent_gb300 as bsfp8

    c = s["case"]
    op, M = c["op"], c["rows"]
    if op == "product":
        bsfp8.bs16_grouped_gemm(s["A"], s["B"], s["offsets"], s["C"], M, c["N"], c["K"], c["experts"], c["experts"], transposed=c["transposed"])
        return s["C"]
    if op == "wgrad":
        bsfp8.bs16_grouped_wgrad(s["dC"], s["A"], s["offsets"], s["dB"], M, c["N"], c["K"], c["experts"], add=s["add"])
        return s["dB"]
    if op == "wgrad8":
        bsfp8.bsfp8_grouped_wgrad(s["dC"], s["A"], s["dc_scales"], s["a_scales"], s["offsets"], s["dB"], M, c["N"], c["K"], c["experts"], add=s["add"])
        return s["dB"]
    if op == "columns":
        slots = M * max(c["top_k"], 1)
        bsfp8.bsfp8_quantize_columns(s["x"], s["offsets"], s["q"], s["scales"], slots, c["K"], c["experts"], slot_of_row=s["slot_of_row"],
                                     top_k=max(c["top_k"], 1))
        return {"q": s["q"].view(E4M3), "scales": s["scales"]}
    bsfp8.bsmx_swiglu_backward(s["h"], s["d_act"], M, c["N"], d_h=s["d_h"], act=s["act"], q=s["q"], scales=s["scales"], format="blockwise")
    out = {"d_h": s["d_h"]}
    if c["act"]:
        out["act"] = s["act"]
    if c["quantised"]:
        out["q"], out["scales"] = s["q"].view(E4M3), s["scales"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------------------
def _active(rows, experts):
    """Experts that some row of `rows` chooses, about."""
    return experts * (1 - (1 - 1 / experts) ** rows)


def work(case):
    c = case
    op, M = c["op"], c["rows"]
    if op == "product":
        N, K = c["N"], c["K"]
        return {"bytes": 2 * (M * K + M * N + round(_active(M, c["experts"]) * N * K)), "flops": 2 * M * N * K}
    if op in ("wgrad", "wgrad8"):
        N, K, E = c["N"], c["K"], c["experts"]
        kept = M - int(M * c["dropped"])
        out = (4 if c["out"] == "fp32" else 2) * (2 if c["add"] else 1) * E * N * K
        rows = 2 * kept * (N + K) if op == "wgrad" else kept * (N + K) + 4 * (kept // BLOCK + round(_active(kept, E) / 2)) * (N + K)
        return {"bytes": rows + out, "flops": 2 * kept * N * K}
    if op == "columns":
        K, slots = c["K"], M * max(c["top_k"], 1)
        kept = slots - int(slots * c["dropped"])
        read = 2 * K * (round(M * (1 - c["dropped"] ** c["top_k"])) if c["top_k"] else kept) + (4 * kept if c["top_k"] else 0)
        return {"bytes": read + kept * K + 4 * K * (kept // BLOCK + round(_active(kept, c["experts"]) / 2)), "flops": 3 * kept * K}
    n = M * c["N"]
    return {"bytes": 10 * n + (2 * n if c["act"] else 0) + (2 * n + n // 16 if c["quantised"] else 0), "flops": 14 * n}


def _e4m3(v):
    """64-bit values rounded to the nearest e4m3 value, ties to even, at most 448."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_scale(amax):
    return torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)


def exact(case, seed):
    s, c = prepare(case, seed), case
    op, M = c["op"], c["rows"]
    if op == "swiglu_grad":
        gate, up = s["h"].double().chunk(2, dim=1)
        d, sig = s["d_act"].double(), torch.special.expit(gate)
        d_h = torch.cat([d * up * (sig + gate * sig * torch.special.expit(-gate)), d * gate * sig], dim=1)
        out = {"d_h": d_h}
        if c["act"]:
            out["act"] = gate * sig * up
        if c["quantised"]:
            b = d_h.view(M, -1, BLOCK)
            scale = _exact_scale(torch.maximum(b.amax(-1), -b.amin(-1)))
            out["q"], out["scales"] = _e4m3(b / scale[..., None]).view(M, -1), scale.t().contiguous()
        return out
    off = s["offsets"].tolist()
    E = c["experts"]
    if op == "columns":
        slots = M * max(c["top_k"], 1)
        q = torch.zeros(slots, c["K"], dtype=torch.float64, device="cuda")
        scales = torch.zeros(slots // BLOCK + E, c["K"], dtype=torch.float64, device="cuda")
        for e in range(E):
            for j, r in enumerate(range(off[e], off[e + 1], BLOCK)):
                end = min(r + BLOCK, off[e + 1])
                x = s["x"][r:end] if not c["top_k"] else s["x"][s["slot_of_row"][r:end].long().div(c["top_k"], rounding_mode="floor")]
                x = x.double()
                scale = _exact_scale(x.abs().max(0).values)
                q[r:end], scales[off[e] // BLOCK + e + j] = _e4m3(x / scale), scale
        return {"q": q, "scales": scales}
    if op == "product":
        C = torch.zeros(M, c["N"], dtype=torch.float64, device="cuda")
        for e in range(E):
            if off[e + 1] > off[e]:
                B = s["B"][e].double()
                C[off[e]: off[e + 1]] = s["A"][off[e]: off[e + 1]].double() @ (B if c["transposed"] else B.t())
        return C
    dB = torch.zeros(E, c["N"], c["K"], dtype=torch.float64, device="cuda") if s["add"] is None else s["add"].double()

    def values(x, scales, e):
        x = x[off[e]: off[e + 1]]
        if op == "wgrad":
            return x.double()
        first = off[e] // BLOCK + e
        n = x.shape[0]
        return x.view(E4M3).double() * scales[first: first + -(-n // BLOCK)].double().repeat_interleave(BLOCK, 0)[:n]

    for e in range(E):
        if off[e + 1] > off[e]:
            dB[e] += values(s["dC"], s.get("dc_scales"), e).t() @ values(s["A"], s.get("a_scales"), e)
    return dB
