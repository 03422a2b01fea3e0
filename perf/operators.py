"""The operators around the grouped GEMM of a mixture-of-experts layer, as measured cases.

Each case is one pass through one operator of the layer

    residual + RMS norm (quantised)  ->  tokens sorted by expert, quantised into the GEMM's A
    ->  grouped GEMM  ->  SwiGLU (quantised)  ->  grouped GEMM  ->  weighted sum per token

in its plain form (elementary torch operations in fp32, each output rounded once) or, with
`own` set, through the framework's entry points.  e4m3 operands come back as float8 values
beside their scales (fp32, or UE8M0 powers of two); fp4 operands come back through the
product that reads them.
"""
import math

import torch

own = False

SEED_MIX = 1_000_003
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6
# e2m1 magnitudes by code and the midpoints between neighbours; a tie goes to the even code
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a decode step of a few sequences: latency of one launch
        {"name": "norm decode", "op": "norm", "rows": 8, "K": 7168, "format": "mxfp8", "residual": "bf16", "y": True},
        # a prefill chunk that ends at an odd token, residual stream kept in fp32
        {"name": "norm prefill", "op": "norm", "rows": 16381, "K": 8192, "format": "blockwise", "residual": "fp32", "y": False},
        # routing of a decode batch: sort by expert and the GEMM's A
        {"name": "route decode", "op": "route", "rows": 16, "K": 7168, "top_k": 8, "experts": 128, "format": "mxfp8", "dropped": 0.0},
        # routing of a prefill batch with skewed experts; a tenth of the slots belongs to other ranks or is padding
        {"name": "route prefill", "op": "route", "rows": 8192, "K": 7168, "top_k": 8, "experts": 64, "format": "blockwise", "dropped": 0.1},
        # the way back of a decode batch, the residual added
        {"name": "combine decode", "op": "combine", "rows": 61, "N": 4096, "top_k": 8, "experts": 128, "weighted": True, "residual": True, "dropped": 0.0},
        # the way back of a prefill batch
        {"name": "combine prefill", "op": "combine", "rows": 8192, "N": 7168, "top_k": 8, "experts": 64, "weighted": True, "residual": False, "dropped": 0.1},
        # gradient of the weighted sum: a short fine-tuning sequence, and a training batch
        {"name": "combine grad short", "op": "combine_grad", "rows": 77, "N": 2048, "top_k": 2, "experts": 8, "dropped": 0.0},
        {"name": "combine grad", "op": "combine_grad", "rows": 4096, "N": 7168, "top_k": 8, "experts": 64, "dropped": 0.0},
        # the activation between the two products: a decode batch over 128 experts, and a prefill batch
        {"name": "swiglu decode", "op": "swiglu", "rows": 2091, "N": 2048, "format": "mxfp8"},
        {"name": "swiglu prefill", "op": "swiglu", "rows": 65536, "N": 2048, "format": "blockwise"},
        # activations to 4 bits and the product with 4-bit weights: decode, and prefill
        {"name": "fp4 decode", "op": "fp4", "rows": 5, "experts": 8, "N": 4096, "K": 7168, "format": "nvfp4"},
        {"name": "fp4 prefill", "op": "fp4", "rows": 512, "experts": 8, "N": 4096, "K": 7168, "format": "mxfp4"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    w = 128 * rng.randint(lo // 128, hi // 128)
    return w + 128 if w == 3072 else w


def draw(rng):
    op = rng.choice(["norm", "route", "combine", "combine_grad", "swiglu", "fp4"])
    if op == "norm":
        K = _width(rng, 512, 8192)
        return {"op": op, "rows": _log_int(rng, 1, 16381), "K": K, "format": rng.choice(["mxfp8", "blockwise"]),
                "residual": rng.choice(["none", "bf16", "fp32"]), "y": rng.random() < 0.5}
    if op == "route":
        top_k = rng.choice([1, 2, 4, 6, 8])
        return {"op": op, "rows": _log_int(rng, 1, 8192), "K": _width(rng, 512, 7168), "top_k": top_k,
                "experts": rng.choice([8, 60, 64, 128, 256]), "format": rng.choice(["mxfp8", "blockwise"]),
                "dropped": rng.choice([0.0, 0.1, 0.5])}
    if op == "combine":
        return {"op": op, "rows": _log_int(rng, 1, 8192), "N": _width(rng, 512, 7168), "top_k": rng.choice([1, 2, 4, 6, 8]),
                "experts": rng.choice([8, 60, 64, 128, 256]), "weighted": rng.random() < 0.7, "residual": rng.random() < 0.5,
                "dropped": rng.choice([0.0, 0.1, 0.5])}
    if op == "combine_grad":
        return {"op": op, "rows": _log_int(rng, 1, 4096), "N": _width(rng, 512, 7168), "top_k": rng.choice([1, 2, 4, 6, 8]),
                "experts": rng.choice([8, 60, 64, 128, 256]), "dropped": rng.choice([0.0, 0.1])}
    if op == "swiglu":
        return {"op": op, "rows": _log_int(rng, 1, 32768), "N": _width(rng, 512, 4096), "format": rng.choice(["mxfp8", "blockwise"])}
    fmt = rng.choice(["mxfp4", "nvfp4"])
    return {"op": op, "rows": _log_int(rng, 1, 512), "experts": rng.choice([1, 4, 8]), "N": _width(rng, 512, 4096),
            "K": _width(rng, 512, 7168), "format": fmt}


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


def _routing(g, rows, top_k, experts, dropped):
    """(ids int32 [rows, top_k], weights fp32): distinct experts per token by Zipf's law; a
    share `dropped` of the slots, whole tokens among them, is marked -1."""
    p = -torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    p = p[torch.randperm(experts, device="cuda", generator=g)]
    noise = -torch.log(-torch.log(torch.rand(rows, experts, device="cuda", generator=g).clamp_(1e-9, 1 - 1e-7)))
    top, ids = torch.topk(p + noise, top_k, dim=1)
    weights = torch.softmax(top, dim=1)
    ids = ids.to(torch.int32)
    if dropped:
        ids[torch.rand(rows, top_k, device="cuda", generator=g) < dropped / 2] = -1
        ids[torch.rand(rows, device="cuda", generator=g) < dropped / 2] = -1
    return ids.contiguous(), weights.contiguous()


def _places(ids, experts):
    """The row of every slot once the slots are sorted by expert, -1 for dropped ones."""
    flat = ids.reshape(-1).long()
    order = torch.argsort(torch.where(flat < 0, experts, flat), stable=True)
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device="cuda")
    return torch.where(flat < 0, -1, place).to(torch.int32).contiguous()


def _fp4_weights(g, experts, N, K, fmt):
    """Packed e2m1 codes [E, N, K/2] of normal values and scale codes [E, N, K/vec]."""
    v = torch.randn(experts, N, K, device="cuda", generator=g).mul_(2.3)
    mid = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device="cuda")
    code = torch.bucketize(v.abs(), mid).to(torch.uint8)
    code += (v < 0).to(torch.uint8) * 8
    packed = (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous()
    vec = 16 if fmt == "nvfp4" else 32
    shape = (experts, N, K // vec)
    if fmt == "nvfp4":  # e4m3 codes of 0.02 .. 0.08
        scales = (0.02 + 0.06 * torch.rand(shape, device="cuda", generator=g)).to(E4M3).view(torch.uint8)
    else:  # 2^-6 .. 2^-4
        scales = torch.randint(121, 124, shape, device="cuda", generator=g, dtype=torch.uint8)
    return packed, scales.contiguous()


def _scale_buffer(fmt, rows, K):
    if fmt == "blockwise":
        return torch.zeros(K // 128, rows, device="cuda")
    return torch.zeros(rows, K // (16 if fmt == "nvfp4" else 32), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    """Inputs, and the buffers that a program allocates once."""
    g, c = _gen(seed), dict(case)
    s = {"case": c}
    u8 = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    if c["op"] == "norm":
        T, K = c["rows"], c["K"]
        s["x"] = _activations(g, T, K)
        s["weight"] = (1 + 0.2 * torch.randn(K, device="cuda", generator=g)).to(torch.bfloat16)
        if c["residual"] != "none":
            dtype = torch.bfloat16 if c["residual"] == "bf16" else torch.float32
            s["residual"] = _activations(g, T, K, dtype, 2.0)
            s["residual_out"] = torch.empty_like(s["residual"])
        s["y_out"] = torch.empty_like(s["x"]) if c["y"] else None
        s["q"], s["scales"] = u8(T, K), _scale_buffer(c["format"], T, K)
    elif c["op"] == "route":
        T, K, k, E = c["rows"], c["K"], c["top_k"], c["experts"]
        s["x"] = _activations(g, T, K)
        s["ids"], _ = _routing(g, T, k, E, c["dropped"])
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        s["offsets"], s["row_of_slot"], s["slot_of_row"] = i32(E + 2), i32(T * k), i32(T * k)
        s["workspace"] = u8(4 * (E + 1) * 256 + 4096)
        s["q"], s["scales"] = u8(T * k, K), _scale_buffer(c["format"], T * k, K)
    elif c["op"] in ("combine", "combine_grad"):
        T, N, k, E = c["rows"], c["N"], c["top_k"], c["experts"]
        ids, s["weights"] = _routing(g, T, k, E, c["dropped"])
        s["row_of_slot"] = _places(ids, E)
        s["C"] = _activations(g, T * k, N, spread=0.3)
        if c["op"] == "combine":
            s["residual"] = _activations(g, T, N) if c["residual"] else None
            s["out"] = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        else:
            s["d_out"] = _activations(g, T, N, spread=0.01)
            s["dC"], s["d_weights"] = torch.zeros_like(s["C"]), torch.empty(T, k, device="cuda")
    elif c["op"] == "swiglu":
        M, N = c["rows"], c["N"]
        s["h"] = _activations(g, M, 2 * N)
        s["q"], s["scales"] = u8(M, N), _scale_buffer(c["format"], M, N)
    else:
        E, m, N, K, fmt = c["experts"], c["rows"], c["N"], c["K"], c["format"]
        s["x"] = _activations(g, E * m, K)
        s["B"], s["b_scales"] = _fp4_weights(g, E, N, K, fmt)
        s["offsets"] = torch.arange(0, E * m + 1, m, dtype=torch.int32, device="cuda")
        s["q"], s["scales"] = u8(E * m, K // 2), _scale_buffer(fmt, E * m, K)
        s["C"] = torch.empty(E * m, N, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
def _power_scale(amax, top):
    """The smallest 2^j with amax / 2^j <= top, as (UE8M0 code, 2^-j); code 127 for zeros."""
    mant, expo = torch.frexp(amax)  # amax = mant * 2^expo, 0.5 <= mant < 1; top = 1.75 * 2^8 or 1.5 * 2^2
    lead, at = (0.875, 9) if top == 448.0 else (0.75, 3)
    j = expo - at + (mant > lead).to(expo.dtype)
    code = torch.where(amax > 0, (j + 127).clamp(0, 254), 127)
    return code.to(torch.uint8), torch.exp2((127 - code).float())


def _to_e4m3(v):
    return v.clamp(-448.0, 448.0).to(E4M3)


def _quantise(v, fmt):
    """(float8 codes, scales) of fp32 rows."""
    rows, K = v.shape
    if fmt == "blockwise":
        b = v.reshape(rows, K // 128, 128)
        amax = b.abs().amax(-1)
        scale = torch.where(amax > 0, (amax / 448.0).clamp(min=2.0 ** -126), 1.0)
        return _to_e4m3(b * (1.0 / scale).unsqueeze(-1)).reshape(rows, K), scale.t().contiguous()
    b = v.reshape(rows, K // 32, 32)
    code, inv = _power_scale(b.abs().amax(-1), 448.0)
    return _to_e4m3(b * inv.unsqueeze(-1)).reshape(rows, K), code.view(E8M0)


def _quantise_fp4(v, fmt):
    """fp32 rows rounded to e2m1 under their block scales, as the values they then stand for."""
    rows, K = v.shape
    vec = 16 if fmt == "nvfp4" else 32
    b = v.reshape(rows, K // vec, vec)
    amax = b.abs().amax(-1)
    if fmt == "nvfp4":
        scale = (amax / 6.0).clamp(2.0 ** -9, 448.0).to(E4M3).float()
        scale = torch.where(amax > 0, scale, 1.0)
        m = (b / scale.unsqueeze(-1)).abs()
    else:
        code, inv = _power_scale(amax, 6.0)
        scale = torch.exp2(code.float() - 127)
        m = (b * inv.unsqueeze(-1)).abs()
    code = ((m > 0.25).long() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    value = torch.tensor(E2M1, device=v.device)[code]
    return (torch.copysign(value, b) * scale.unsqueeze(-1)).reshape(rows, K)


def _unpack_fp4(packed, scales, fmt):
    table = torch.tensor(E2M1 + tuple(-m for m in E2M1), device=packed.device)
    codes = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2)
    s = scales.view(E4M3).float() if fmt == "nvfp4" else torch.exp2(scales.float() - 127)
    return table[codes.long()] * s.repeat_interleave(16 if fmt == "nvfp4" else 32, dim=-1)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        h = s["x"].float()
        if c["residual"] != "none":
            h = h + s["residual"].float()
        n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
        q, scales = _quantise(n, c["format"])
        out = {"q": q, "scales": scales}
        if c["residual"] != "none":
            out["residual"] = h.to(s["residual"].dtype)
        if c["y"]:
            out["y"] = n.to(torch.bfloat16)
        return out
    if c["op"] == "route":
        T, k, E = c["rows"], c["top_k"], c["experts"]
        flat = s["ids"].reshape(-1).long()
        key = torch.where((flat >= 0) & (flat < E), flat, E)
        key, order = torch.sort(key, stable=True)
        offsets = torch.searchsorted(key, torch.arange(E + 2, device="cuda")).to(torch.int32)
        kept = key < E
        slot_of_row = torch.where(kept, order, -1).to(torch.int32)
        row_of_slot = torch.empty_like(slot_of_row)
        row_of_slot[order] = torch.where(kept, torch.arange(T * k, device="cuda"), -1).to(torch.int32)
        q, scales = _quantise(s["x"].float(), c["format"])
        token = order // k  # a dropped slot leaves a row of zeros
        q = torch.where(kept[:, None], q.view(torch.uint8)[token], 0).view(E4M3)
        if c["format"] == "blockwise":
            scales = torch.where(kept, scales[:, token], 0.0)
        else:
            scales = torch.where(kept[:, None], scales.view(torch.uint8)[token], 0).view(E8M0)
        return {"offsets": offsets, "row_of_slot": row_of_slot, "slot_of_row": slot_of_row, "q": q, "scales": scales}
    if c["op"] in ("combine", "combine_grad"):
        T, N, k = c["rows"], c["N"], c["top_k"]
        row = s["row_of_slot"].long()
        live = (row >= 0)[:, None]
        C = torch.where(live, s["C"][row.clamp(min=0)].float(), 0.0).reshape(T, k, N)
        if c["op"] == "combine":
            out = (C * s["weights"][:, :, None]).sum(1) if c["weighted"] else C.sum(1)
            if c["residual"]:
                out = out + s["residual"].float()
            return out.to(torch.bfloat16)
        d_out = s["d_out"].float()
        d_weights = (C * d_out[:, None, :]).sum(-1)
        dC = torch.zeros_like(s["C"])
        d_slot = (d_out[:, None, :] * s["weights"][:, :, None]).reshape(T * k, N).to(torch.bfloat16)
        kept = row[row >= 0]
        dC[kept] = d_slot[row >= 0]
        return {"dC": dC, "d_weights": d_weights}
    if c["op"] == "swiglu":
        gate, up = s["h"][:, : c["N"]].float(), s["h"][:, c["N"]:].float()
        q, scales = _quantise(gate / (1 + torch.exp(-gate)) * up, c["format"])
        return {"q": q, "scales": scales}
    E, m, K = c["experts"], c["rows"], c["K"]
    a = _quantise_fp4(s["x"].float(), c["format"]).reshape(E, m, K)
    w = _unpack_fp4(s["B"], s["b_scales"], c["format"])
    return torch.bmm(a, w.transpose(1, 2)).reshape(E * m, c["N"]).to(torch.bfloat16)


def _own(s):
    import block_scaled_fp8_persistent_gb300 as bsfp8

    c = s["case"]
    if c["op"] == "norm":
        residual_out = s.get("residual_out")
        bsfp8.bsmx_rmsnorm_quant(c["format"], s["x"], s["weight"], EPS, c["rows"], c["K"], residual=s.get("residual"),
                                 residual_out=residual_out, y=s["y_out"], q=s["q"], scales=s["scales"])
        out = {"q": s["q"].view(E4M3), "scales": s["scales"] if c["format"] == "blockwise" else s["scales"].view(E8M0)}
        if residual_out is not None:
            out["residual"] = residual_out
        if c["y"]:
            out["y"] = s["y_out"]
        return out
    if c["op"] == "route":
        T, k = c["rows"], c["top_k"]
        bsfp8.bsmx_moe_sort(s["ids"], s["offsets"], s["row_of_slot"], s["workspace"], T, k, c["experts"], slot_of_row=s["slot_of_row"])
        bsfp8.bsmx_quantize(c["format"], s["x"], s["q"], s["scales"], T, c["K"], row_of_slot=s["row_of_slot"], top_k=k, out_rows=T * k)
        return {"offsets": s["offsets"], "row_of_slot": s["row_of_slot"], "slot_of_row": s["slot_of_row"], "q": s["q"].view(E4M3),
                "scales": s["scales"] if c["format"] == "blockwise" else s["scales"].view(E8M0)}
    if c["op"] == "combine":
        T, k = c["rows"], c["top_k"]
        bsfp8.bsmx_moe_combine(s["C"], s["row_of_slot"], s["out"], T, T * k, k, c["N"], weights=s["weights"] if c["weighted"] else None,
                               residual=s["residual"])
        return s["out"]
    if c["op"] == "combine_grad":
        T, k = c["rows"], c["top_k"]
        bsfp8.bsmx_moe_combine_backward(s["d_out"], s["C"], s["row_of_slot"], s["weights"], s["dC"], s["d_weights"], T, T * k, k, c["N"])
        return {"dC": s["dC"], "d_weights": s["d_weights"]}
    if c["op"] == "swiglu":
        bsfp8.bsmx_swiglu_quant(c["format"], s["h"], s["q"], s["scales"], c["rows"], c["N"])
        return {"q": s["q"].view(E4M3), "scales": s["scales"] if c["format"] == "blockwise" else s["scales"].view(E8M0)}
    E, M, fmt = c["experts"], c["experts"] * c["rows"], c["format"]
    bsfp8.bsmx_quantize(fmt, s["x"], s["q"], s["scales"], M, c["K"])
    bsfp8.bsmx_grouped_gemm(fmt, fmt, s["q"], s["B"], s["scales"], s["b_scales"], s["offsets"], s["C"], M, c["N"], c["K"], E, E)
    return s["C"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------------------
def _quantised_bytes(fmt, rows, K):
    return {"blockwise": rows * K + rows * K // 32, "mxfp8": rows * K + rows * K // 32,
            "mxfp4": rows * K // 2 + rows * K // 32, "nvfp4": rows * K // 2 + rows * K // 16}[fmt]


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["K"]
        res = {"none": 0, "bf16": 4, "fp32": 8}[c["residual"]]
        return {"bytes": n * (2 + res + (2 if c["y"] else 0)) + 2 * c["K"] + _quantised_bytes(c["format"], c["rows"], c["K"]), "flops": 7 * n}
    if c["op"] == "route":
        slots = c["rows"] * c["top_k"]
        kept = round(slots * (1 - c["dropped"] / 2) ** 2)
        return {"bytes": 12 * slots + 4 * c["experts"] + 2 * c["rows"] * c["K"] + _quantised_bytes(c["format"], kept, c["K"]),
                "flops": 3 * c["rows"] * c["K"]}
    if c["op"] in ("combine", "combine_grad"):
        T, N, slots = c["rows"], c["N"], c["rows"] * c["top_k"]
        kept = round(slots * (1 - c["dropped"] / 2) ** 2)
        if c["op"] == "combine":
            return {"bytes": 2 * N * (kept + T + (T if c["residual"] else 0)) + slots * (8 if c["weighted"] else 4), "flops": 2 * kept * N}
        return {"bytes": 2 * N * (2 * kept + T) + 12 * slots, "flops": 3 * kept * N}
    if c["op"] == "swiglu":
        n = c["rows"] * c["N"]
        return {"bytes": 4 * n + _quantised_bytes(c["format"], c["rows"], c["N"]), "flops": 8 * n}
    E, M, N, K, fmt = c["experts"], c["experts"] * c["rows"], c["N"], c["K"], c["format"]
    return {"bytes": 2 * M * K + _quantised_bytes(fmt, E * N, K) + 2 * M * N, "flops": 2 * M * N * K}


def _near(v, bits, low, top):
    """64-bit values rounded to the nearest with `bits` fraction bits, multiples of 2^(low - bits)
    below 2^low, ties to even, at most `top`."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=low).double() - bits)
    return (torch.round(v / step) * step).clamp(-top, top)


def _exact_quantised(v, fmt):
    """(codes' values, scales) per format, blocks along the rows, from 64-bit values."""
    rows, K = v.shape
    vec = {"blockwise": 128, "mxfp8": 32, "mxfp4": 32, "nvfp4": 16}[fmt]
    top = 6.0 if "fp4" in fmt else 448.0
    b = v.view(rows, K // vec, vec)
    amax = torch.maximum(b.amax(-1), -b.amin(-1))
    if fmt == "blockwise":
        scale = amax / top
    elif fmt == "nvfp4":
        scale = _near((amax / top).clamp(min=2.0 ** -9), 3, -6, 448.0)
    else:
        j = torch.ceil(torch.log2(amax / top)).clamp(-127, 127)
        scale = torch.exp2(j - (amax <= top * torch.exp2(j - 1)).double())  # the logarithm of a power of two may round up
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    q = _near(b / scale[..., None], 1, 0, top) if "fp4" in fmt else _near(b / scale[..., None], 3, -6, top)
    return q.view(rows, K), scale


def exact(case, seed):
    s, c = prepare(case, seed), case
    lay = lambda scale, fmt: scale.t().contiguous() if fmt == "blockwise" else scale  # noqa: E731
    if c["op"] == "norm":
        h = s["x"].double()
        if c["residual"] != "none":
            h += s["residual"].double()
        n = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / c["K"] + EPS) * s["weight"].double()
        q, scale = _exact_quantised(n, c["format"])
        out = {"q": q, "scales": lay(scale, c["format"])}
        if c["residual"] != "none":
            out["residual"] = h
        if c["y"]:
            out["y"] = n
        return out
    if c["op"] == "route":
        q, scale = _exact_quantised(s["x"].double(), c["format"])
        place = _places(s["ids"], c["experts"]).long()
        slot = torch.nonzero(place >= 0).squeeze(1)
        slots = c["rows"] * c["top_k"]
        rows = torch.zeros(slots, c["K"], dtype=torch.float64, device="cuda")
        rows[place[slot]] = q[slot // c["top_k"]]
        scales = torch.zeros(slots, scale.shape[1], dtype=torch.float64, device="cuda")
        if c["format"] == "mxfp8":
            scales += 2.0 ** -127  # code 0
        scales[place[slot]] = scale[slot // c["top_k"]]
        return {"offsets": None, "row_of_slot": None, "slot_of_row": None, "q": rows, "scales": lay(scales, c["format"])}
    if c["op"] in ("combine", "combine_grad"):
        T, k, N = c["rows"], c["top_k"], c["N"]
        row = s["row_of_slot"].view(T, k).long()
        grad = c["op"] == "combine_grad"
        acc = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        if not grad and c["residual"]:
            acc += s["residual"].double()
        dC = torch.zeros(T * k, N, dtype=torch.float64, device="cuda") if grad else None
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(row[:, j] >= 0).squeeze(1)
            r, w = row[t, j], s["weights"][t, j].double()[:, None]
            if grad:
                d = s["d_out"][t].double()
                dC[r] = d * w
                dw[t, j] = torch.einsum("tn,tn->t", d, s["C"][r].double())
            else:
                acc[t] += s["C"][r].double() * (w if c["weighted"] else 1.0)
        return {"dC": dC, "d_weights": dw} if grad else acc
    if c["op"] == "swiglu":
        gate, up = s["h"].double().chunk(2, dim=1)
        q, scale = _exact_quantised(gate * torch.special.expit(gate) * up, c["format"])
        return {"q": q, "scales": lay(scale, c["format"])}
    E, m, N, K, fmt = c["experts"], c["rows"], c["N"], c["K"], c["format"]
    q, scale = _exact_quantised(s["x"].double(), fmt)
    a = (q.view(E * m, -1, K // scale.shape[1]) * scale[..., None]).reshape(E, m, K)
    code = torch.stack([s["B"] % 16, s["B"] // 16], dim=-1).reshape(E, N, K).long()
    level, sign = code % 8, 1.0 - 2.0 * (code // 8).double()
    value = torch.where(level < 2, level / 2.0, (1.0 + (level % 2) / 2.0) * torch.exp2((level // 2 - 1).double())) * sign
    b_scale = s["b_scales"].view(E4M3).double() if fmt == "nvfp4" else torch.exp2(s["b_scales"].double() - 127)
    w = (value.view(E, N, -1, K // b_scale.shape[-1]) * b_scale[..., None]).reshape(E, N, K)
    return torch.stack([a[e] @ w[e].t() for e in range(E)]).reshape(E * m, N)
