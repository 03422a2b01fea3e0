"""The operators around the grouped GEMM on the GPU against their 64-bit definitions
(moe_reference.py).

Tolerances, each from the arithmetic and set before the first run (2^-24 = one fp32 rounding):
  quantisation    exact for the MX formats (the scale is a power of two) and, of 16-bit inputs,
                  for nvfp4's elements (the quotient is rounded once, ties are exact); nvfp4's
                  scale and fp32 inputs 2^-23, blockwise 2^-22 (reciprocal and product)
  norm            2^-18: sums of at most 32 + 10 terms per thread and step, a reciprocal square
                  root of 2 ulp and three products; bf16 outputs half a bf16 ulp more
  SwiGLU          (8 + |g|) * 2^-22: the exponential's argument is rounded to 2^-24 |g| log2(e)
  combine         (top_k + 1) * 2^-24 of the sum of magnitudes and half a bf16 ulp
  its gradient    d_weights: 8 terms per 2048 columns in a thread, 5 shuffles, 8 warps, doubled
"""
import threading

import numpy as np
import pytest
import torch

import block_scaled_fp8_persistent_gb300 as bsfp8
import moe_reference as ref

pytestmark = pytest.mark.gpu

FORMATS = ["mxfp8", "mxfp4", "nvfp4", "blockwise"]
ROWS_ERROR = 11
HALF_BF16 = 2.0 ** -8  # a bf16 value is within 2^-9 of what it rounds; doubled for the binade


def _scale_shape(fmt, rows, K):
    return (K // 128, rows) if fmt == "blockwise" else (rows, K // ref.VEC[fmt])


def _operand(fmt, rows, K, fill=0):
    """(q, scales) with two guard rows' worth of bytes behind each, filled with `fill`."""
    width = K // 2 if "fp4" in fmt else K
    q = torch.full(((rows + 2) * width,), fill, dtype=torch.uint8, device="cuda")
    n = rows * K // ref.VEC[fmt]
    if fmt == "blockwise":
        s = torch.full((n + 64,), float(fill), device="cuda")
    else:
        s = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
    return q, s


def _check_guards(fmt, q, s, rows, K, fill):
    width = K // 2 if "fp4" in fmt else K
    assert torch.all(q[rows * width:] == fill)
    assert torch.all(s[rows * K // ref.VEC[fmt]:] == fill)


def _check(fmt, v, q, s, rows, K, u_value, u_scale):
    width = K // 2 if "fp4" in fmt else K
    ref.check_quantised(v, q[: rows * width], s[: rows * K // ref.VEC[fmt]], fmt, u_value, u_scale)


def _rand(shape, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[0], 1, generator=g))
    return x.to(dtype)


def _u(fmt, dtype):
    if fmt in ("mxfp8", "mxfp4"):
        return 0.0, 0.0
    if fmt == "nvfp4":
        return (0.0 if dtype != torch.float32 else 2.0 ** -23), 2.0 ** -23
    return 2.0 ** -22, 2.0 ** -22


def _no_error():
    assert bsfp8.bsfp8_get_device_error() == 0


# ------------------------------------------------------------------------------ quantise
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 128), (9, 128), (11, 256), (7, 384), (3, 640), (5, 1024), (37, 1152),
                                    (130, 7168), (2, 16512)])
def test_quantize(fmt, dtype, rows, K):
    x = _rand((rows, K), dtype, seed=K + rows, spread=1.0 if dtype == torch.float16 else 3.0)
    x[0, :32] = 0
    x[rows - 1, -128:] = 0
    q, s = _operand(fmt, rows, K, fill=7)
    bsfp8.bsmx_quantize(fmt, x.cuda(), q, s, rows, K)
    _no_error()
    _check(fmt, x.double().numpy(), q, s, rows, K, *_u(fmt, dtype))
    _check_guards(fmt, q, s, rows, K, 7)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_every_scale(fmt):
    # block maxima over bf16's whole range, subnormal to largest, each with ties in the block
    lead = torch.arange(1, 0x7F80, 37, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    rows, K = len(lead), 128
    step = torch.tensor([1, 0.5, 0.25, 0.75, 0.4375, 0.21875, 1 / 12, -1 / 6, -0.125, 0.0625, -0.28125, 0])
    x = (lead.double()[:, None] * step.double().repeat(11)[:K][None, :]).to(torch.bfloat16)
    x[:, 0:K:16] = lead[:, None]
    q, s = _operand(fmt, rows, K)
    bsfp8.bsmx_quantize(fmt, x.cuda(), q, s, rows, K)
    v = x.double().numpy()
    if fmt == "blockwise":  # products with subnormal results round at 2^-149, not relatively
        keep = lead.double().numpy() > 1e-30
        width = K
        ref.check_quantised(v[keep], q[: rows * width].view(rows, width)[torch.from_numpy(keep).cuda()],
                            s[: rows].view(1, rows)[:, torch.from_numpy(keep).cuda()], fmt, *_u(fmt, torch.bfloat16))
    else:
        _check(fmt, v, q, s, rows, K, *_u(fmt, torch.bfloat16))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantize_non_finite_blocks_have_nan_scales(fmt, bad):
    rows, K = 4, 512
    x = _rand((rows, K), torch.bfloat16, seed=2, spread=0.1)
    clean, clean_s = _operand(fmt, rows, K)
    bsfp8.bsmx_quantize(fmt, x.cuda(), clean, clean_s, rows, K)
    x[2, 200] = bad
    q, s = _operand(fmt, rows, K)
    bsfp8.bsmx_quantize(fmt, x.cuda(), q, s, rows, K)
    width, vec = (K // 2 if "fp4" in fmt else K), ref.VEC[fmt]
    sc = ref.decode(q[: rows * width], s[: rows * K // vec], fmt, rows, K)[1]
    hit = np.zeros_like(sc, bool)
    hit[2, 200 // vec] = True
    assert np.isnan(sc[hit]).all() and np.isfinite(sc[~hit]).all()
    same = (q[: rows * width].view(rows, K // vec, -1) == clean[: rows * width].view(rows, K // vec, -1)).all(-1)
    assert same[~torch.from_numpy(hit).cuda()].all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_of_16_byte_aligned_rows(fmt):
    rows, K = 19, 384
    flat = _rand((rows * K + 8, 1), torch.bfloat16, seed=4, spread=0.0).reshape(-1).cuda()
    x = flat[8:].view(rows, K)
    assert x.data_ptr() % 32 == 16
    a, b = _operand(fmt, rows, K), _operand(fmt, rows, K)
    bsfp8.bsmx_quantize(fmt, x, *a, rows, K)
    bsfp8.bsmx_quantize(fmt, x.clone(), *b, rows, K)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,top_k,E,K", [(1, 1, 1, 128), (1, 8, 8, 7168), (5, 3, 4, 640), (67, 8, 16, 1152), (40, 11, 32, 256),
                                               (700, 2, 8, 1152), (513, 3, 8, 128), (520, 1, 4, 9216)])
def test_quantize_by_row_map(fmt, rows, top_k, E, K):
    g = np.random.default_rng(rows * top_k)
    ids = g.integers(-1, E, size=(rows, top_k)).astype(np.int32)
    ids[rows // 2] = -1  # a token that goes nowhere
    _, row, slot = ref.sort_slots(ids, E)
    x = _rand((rows, K), torch.bfloat16, seed=9, spread=1.0).cuda()
    n = rows * top_k
    q, s = _operand(fmt, n, K, fill=9)
    bsfp8.bsmx_quantize(fmt, x, q, s, rows, K, row_of_slot=torch.from_numpy(row).cuda(), top_k=top_k, out_rows=n)
    _no_error()
    width, vec = (K // 2 if "fp4" in fmt else K), ref.VEC[fmt]
    pq, ps = _operand(fmt, rows, K)
    bsfp8.bsmx_quantize(fmt, x, pq, ps, rows, K)
    live = torch.from_numpy(slot >= 0).cuda()
    token = torch.from_numpy(np.maximum(slot, 0) // top_k).cuda()
    got = q[: n * width].view(n, width)
    assert torch.equal(got[live], pq[: rows * width].view(rows, width)[token[live]])
    assert torch.all(got[~live] == 9)
    if fmt == "blockwise":
        gs, want = s[: n * K // vec].view(-1, n).t(), ps[: rows * K // vec].view(-1, rows).t()
    else:
        gs, want = s[: n * K // vec].view(n, -1), ps[: rows * K // vec].view(rows, -1)
    assert torch.equal(gs[live], want[token[live]])
    assert torch.all(gs[~live] == 9)
    _check_guards(fmt, q, s, n, K, 9)


def test_row_map_of_every_slot_by_default():
    rows, top_k, K = 6, 3, 256
    x = _rand((rows, K), torch.bfloat16, seed=4, spread=0.5).cuda()
    row = torch.randperm(rows * top_k, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    q, s = _operand("mxfp8", rows * top_k, K)
    bsfp8.bsmx_quantize("mxfp8", x, q, s, rows, K, row_of_slot=row, top_k=top_k)
    _no_error()
    want_q, want_s = _operand("mxfp8", rows * top_k, K)
    bsfp8.bsmx_quantize("mxfp8", x, want_q, want_s, rows, K, row_of_slot=row, top_k=top_k, out_rows=rows * top_k)
    assert torch.equal(q, want_q) and torch.equal(s, want_s) and torch.all(s[: rows * top_k * K // 32] > 0)


def test_rows_out_of_range_are_recorded_and_skipped():
    rows, K, top_k = 6, 256, 2
    x = _rand((rows, K), torch.bfloat16, seed=1, spread=0.5).cuda()
    row = torch.arange(12, dtype=torch.int32, device="cuda")
    row[7] = 12
    q, s = _operand("mxfp8", 12, K, fill=5)
    bsfp8.bsmx_quantize("mxfp8", x, q, s, rows, K, row_of_slot=row, top_k=top_k, out_rows=12)
    assert bsfp8.bsfp8_get_device_error() == ROWS_ERROR
    assert torch.all(q.view(-1, K)[7] == 5) and not torch.all(q.view(-1, K)[8] == 5)
    _check_guards("mxfp8", q, s, 12, K, 5)
    C = _rand((12, K), torch.bfloat16, seed=1, spread=0.5).cuda()
    w = torch.ones(rows, top_k, device="cuda")
    out, dw = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda"), torch.ones_like(w)
    bsfp8.bsmx_moe_combine(C, row, out, rows, 12, top_k, K, weights=w)
    assert bsfp8.bsfp8_get_device_error() == ROWS_ERROR
    assert torch.equal(out[3], C[6])
    dC = torch.zeros_like(C)
    bsfp8.bsmx_moe_combine_backward(out, C, row, w, dC, dw, rows, 12, top_k, K)
    assert bsfp8.bsfp8_get_device_error() == ROWS_ERROR
    assert dw[3, 1] == 0 and torch.all(dC[7] == 0)
    _no_error()


# ---------------------------------------------------------------------------------- norm
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 128), (70, 128), (9, 256), (13, 512), (7, 640), (5, 1024), (33, 7168), (3, 8320),
                                    (2, 16512), (1, 32768)])
def test_norm(fmt, residual, rows, K):
    x = _rand((rows, K), torch.bfloat16, seed=K, spread=2.0)
    w = (1 + 0.3 * torch.randn(K, generator=torch.Generator().manual_seed(5))).to(torch.bfloat16)
    r = None if residual is None else _rand((rows, K), residual, seed=K + 1, spread=2.0)
    eps = 1e-5
    y = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    ro = None if r is None else torch.empty(rows, K, dtype=residual, device="cuda")
    q, s = _operand(fmt, rows, K, fill=3)
    bsfp8.bsmx_rmsnorm_quant(fmt, x.cuda(), w.cuda(), eps, rows, K, residual=None if r is None else r.cuda(),
                             residual_out=ro, y=y, q=q, scales=s)
    _no_error()
    h = x.double() if r is None else x.double() + r.double()
    n = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()
    u = 2.0 ** -18
    _check(fmt, n.numpy(), q, s, rows, K, u, u)
    _check_guards(fmt, q, s, rows, K, 3)
    assert torch.all((y.cpu().double() - n).abs() <= n.abs() * (HALF_BF16 + u) + 1e-38)
    if r is not None:
        assert torch.equal(ro.cpu(), (x.float() + r.float()).to(residual))


@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32])
def test_norm_in_place_residual_and_single_outputs(residual):
    rows, K = 21, 2048
    x = _rand((rows, K), torch.bfloat16, seed=1).cuda()
    r = _rand((rows, K), residual, seed=2).cuda()
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    ro, y = torch.empty_like(r), torch.empty_like(x)
    q, s = _operand("mxfp8", rows, K)
    bsfp8.bsmx_rmsnorm_quant("mxfp8", x, w, 1e-6, rows, K, residual=r, residual_out=ro, y=y, q=q, scales=s)
    y2, q2, s2 = torch.empty_like(y), *_operand("mxfp8", rows, K)
    bsfp8.bsmx_rmsnorm_quant("mxfp8", x, w, 1e-6, rows, K, residual=r, y=y2)
    bsfp8.bsmx_rmsnorm_quant("mxfp8", x, w, 1e-6, rows, K, residual=r, q=q2, scales=s2)
    assert torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(s, s2)
    mine = r.clone()
    bsfp8.bsmx_rmsnorm_quant("mxfp8", x, w, 1e-6, rows, K, residual=mine, residual_out=mine)
    assert torch.equal(mine, ro)
    first = torch.empty_like(r)  # the first layer: the stream starts as x
    bsfp8.bsmx_rmsnorm_quant("mxfp8", x, w, 1e-6, rows, K, residual_out=first)
    assert torch.equal(first, x.to(residual))


def test_norm_of_zero_and_non_finite_rows():
    rows, K = 4, 512
    x = _rand((rows, K), torch.bfloat16, seed=3, spread=0.2)
    x[1] = 0
    x[2, 77] = float("nan")
    y = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    q, s = _operand("mxfp8", rows, K)
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    bsfp8.bsmx_rmsnorm_quant("mxfp8", x.cuda(), w, 1e-6, rows, K, y=y, q=q, scales=s)
    assert torch.all(y[1] == 0) and torch.isnan(y[2]).all()
    sc = s[: rows * K // 32].view(rows, -1)
    assert torch.all(q.view(-1, K)[1] == 0) and torch.all(sc[1] == 127) and torch.all(sc[2] == 255)
    assert torch.isfinite(y[[0, 3]]).all() and torch.all(sc[[0, 3]] < 255)


@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [128, 640, 9216])
def test_norm_of_16_byte_aligned_rows(residual, K):
    rows = 9

    def buffer(dtype, seed, skip):
        flat = _rand((rows * K + 16, 1), dtype, seed=seed, spread=0.0).reshape(-1).cuda()
        return flat[skip: skip + rows * K].view(rows, K)

    step = 8 if residual == torch.bfloat16 else 4
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    x, r = buffer(torch.bfloat16, 4, 0), buffer(residual, 5, 0)
    want = torch.empty_like(x), torch.empty_like(r)
    bsfp8.bsmx_rmsnorm_quant("mxfp8", x, w, 1e-6, rows, K, residual=r, y=want[0], residual_out=want[1])
    for odd in range(4):  # each buffer in turn off a 32-byte boundary
        bufs = [buffer(torch.bfloat16, 4, 8 * (odd == 0)), buffer(residual, 5, step * (odd == 1)),
                buffer(torch.bfloat16, 6, 8 * (odd == 2)), buffer(residual, 7, step * (odd == 3))]
        bufs[0].copy_(x)
        bufs[1].copy_(r)
        assert bufs[odd].data_ptr() % 32 == 16
        bsfp8.bsmx_rmsnorm_quant("mxfp8", bufs[0], w, 1e-6, rows, K, residual=bufs[1], y=bufs[2], residual_out=bufs[3])
        assert torch.equal(bufs[2], want[0]) and torch.equal(bufs[3], want[1])


# -------------------------------------------------------------------------------- SwiGLU
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,N", [(1, 128), (17, 128), (3, 384), (5, 640), (131, 2048), (3, 9216)])
def test_swiglu(fmt, rows, N):
    h = _rand((rows, 2 * N), torch.bfloat16, seed=N, spread=1.0)
    h[0, :64] = 30.0
    q, s = _operand(fmt, rows, N, fill=4)
    bsfp8.bsmx_swiglu_quant(fmt, h.cuda(), q, s, rows, N)
    _no_error()
    g, u = h[:, :N].double().clamp(-80, None), h[:, N:].double()
    assert torch.equal(g, h[:, :N].double())  # the inputs stay where exp(-g) is finite
    v = g / (1 + torch.exp(-g)) * u
    err = ((8 + g.abs()) * 2.0 ** -22).numpy()
    _check(fmt, v.numpy(), q, s, rows, N, err, 2.0 ** -21)
    _check_guards(fmt, q, s, rows, N, 4)


def test_swiglu_of_extreme_gates():
    N = 256
    h = torch.ones(4, 2 * N, dtype=torch.bfloat16)
    h[0, :N] = -300.0  # exp(300) is past fp32: the product is 0
    h[1, :N] = 300.0
    h[2, 3] = float("inf")
    h[3, N + 130] = float("nan")
    h[3, 0], h[3, N] = -1e20, 1e20  # 0 although gate times up is past fp32
    q, s = _operand("mxfp8", 4, N)
    bsfp8.bsmx_swiglu_quant("mxfp8", h.cuda(), q, s, 4, N)
    v, sc = ref.decode(q[: 4 * N], s[: 4 * N // 32], "mxfp8", 4, N)
    assert np.all(v[0] == 0) and np.all(sc[0] == 1)
    assert np.all(v[1] * sc[1][0] == 288.0)  # 300 = 300 / 1 in e4m3's grid of 32
    assert np.isnan(sc[2, 0]) and np.isfinite(sc[2, 1:]).all()
    assert v[3, 0] == 0
    assert np.isnan(sc[3, 130 // 32]) and np.isfinite(np.delete(sc[3], 130 // 32)).all()


# ---------------------------------------------------------------------------------- sort
def _sort(ids, E, with_slot=True):
    rows, top_k = ids.shape
    n = rows * top_k
    d = torch.from_numpy(ids).cuda()
    off = torch.full((E + 2 + 4,), -7, dtype=torch.int32, device="cuda")
    row = torch.full((n + 4,), -7, dtype=torch.int32, device="cuda")
    slot = torch.full((n + 4,), -7, dtype=torch.int32, device="cuda") if with_slot else None
    ws = torch.full((bsfp8.bsmx_moe_sort_workspace(rows, top_k, E) + 16,), 0xAB, dtype=torch.uint8, device="cuda")
    bsfp8.bsmx_moe_sort(d, off, row, ws, rows, top_k, E, slot_of_row=slot)
    assert torch.all(off[E + 2:] == -7) and torch.all(row[n:] == -7) and torch.all(ws[-16:] == 0xAB)
    if with_slot:
        assert torch.all(slot[n:] == -7)
    return off[: E + 2].cpu().numpy(), row[:n].cpu().numpy(), None if slot is None else slot[:n].cpu().numpy()


@pytest.mark.parametrize("E", [1, 8, 60, 256, 1500, 4096])
@pytest.mark.parametrize("rows,top_k", [(0, 8), (1, 1), (1, 8), (31, 1), (33, 2), (129, 6), (512, 8), (513, 8), (512, 2), (1025, 1), (1024, 4), (700, 11), (2048, 8), (2049, 8),
                                        (5000, 1), (16384, 8), (20011, 9), (70001, 8)])
def test_sort(rows, top_k, E):
    g = np.random.default_rng(rows + E)
    ids = np.minimum(g.zipf(1.3, size=(rows, top_k)) - 1, 1 << 20).astype(np.int32)
    ids[g.random((rows, top_k)) < 0.1] = -1
    got = _sort(ids, E)
    want = ref.sort_slots(ids, E)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("rows", [100, 3000, 9000])
@pytest.mark.parametrize("kind", ["dropped", "one", "last", "wild", "sorted", "reversed"])
def test_sort_extremes(rows, kind):
    E, k = 64, 2
    n = rows * k
    ids = {"dropped": np.full(n, -1), "one": np.full(n, 5), "last": np.full(n, E - 1),
           "wild": np.resize([E, 2 ** 31 - 1, -2 ** 31, 0, E - 1, -1], n),
           "sorted": np.arange(n) * E // n, "reversed": (n - 1 - np.arange(n)) * E // n}[kind]
    ids = ids.astype(np.int32).reshape(rows, k)
    got = _sort(ids, E, with_slot=kind != "one")
    for a, b in zip(got, ref.sort_slots(ids, E)):
        assert a is None or np.array_equal(a, b)


def test_sorts_of_different_sizes_on_two_threads():
    # 512 and 4096 experts want 68 and 160 KB of shared memory: what one call asks for must not
    # take away what the other is about to launch with.  The C entry point directly, which runs
    # without the interpreter lock.
    lib = bsfp8.load_library()
    rows, top_k, steps = 2048, 8, 3000
    n = rows * top_k
    ids = np.random.default_rng(5).integers(0, 512, size=(rows, top_k)).astype(np.int32)
    d = torch.from_numpy(ids).cuda()
    torch.cuda.synchronize()
    refused, rows_of = {}, {}

    def sort(E):
        off = torch.empty(E + 2, dtype=torch.int32, device="cuda")
        rows_of[E] = torch.empty(n, dtype=torch.int32, device="cuda")
        stream = torch.cuda.Stream()
        args = (d.data_ptr(), off.data_ptr(), rows_of[E].data_ptr(), None, None, 0, rows, top_k, E, stream.cuda_stream)
        refused[E] = sum(lib.bsmx_moe_sort(*args) != 0 for _ in range(steps))
        stream.synchronize()

    threads = [threading.Thread(target=sort, args=(E,)) for E in (512, 4096)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert refused == {512: 0, 4096: 0}
    for E in (512, 4096):
        assert np.array_equal(rows_of[E].cpu().numpy(), ref.sort_slots(ids, E)[1])


def test_a_captured_sort_replays_after_a_smaller_one():
    rows, top_k, E = 2048, 8, 4096
    n = rows * top_k
    ids = np.random.default_rng(6).integers(-1, E, size=(rows, top_k)).astype(np.int32)
    d = torch.from_numpy(ids).cuda()
    off, row = torch.empty(E + 2, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    bsfp8.bsmx_moe_sort(d, off, row, None, rows, top_k, E)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsfp8.bsmx_moe_sort(d, off, row, None, rows, top_k, E)
    _sort(ids, 512)
    off.fill_(-7)
    row.fill_(-7)
    graph.replay()
    want = ref.sort_slots(ids, E)
    assert np.array_equal(off.cpu().numpy(), want[0]) and np.array_equal(row.cpu().numpy(), want[1])


@pytest.mark.parametrize("rows,top_k", [(300, 2), (1500, 4), (2500, 8), (16500, 8)])
def test_chained_sorts(rows, top_k):
    # each sort's ids are the rows that the one before it writes, nothing in between
    E, steps, n = 4096, 6, rows * top_k
    ids = np.random.default_rng(rows).integers(0, E, size=n).astype(np.int32)
    bufs = [torch.from_numpy(ids).cuda()] + [torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(steps)]
    off = torch.empty(steps, E + 2, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(4, bsfp8.bsmx_moe_sort_workspace(rows, top_k, E)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for i in range(steps):
        bsfp8.bsmx_moe_sort(bufs[i], off[i], bufs[i + 1], ws, rows, top_k, E)
    for i in range(steps):
        want_off, ids, _ = ref.sort_slots(ids, E)
        assert np.array_equal(off[i].cpu().numpy(), want_off) and np.array_equal(bufs[i + 1].cpu().numpy(), ids)


# ------------------------------------------------------------------- combine and gradient
def _routed(rows, top_k, E, seed, dropped=0.2):
    g = np.random.default_rng(seed)
    ids = g.integers(0, E, size=(rows, top_k)).astype(np.int32)
    ids[g.random((rows, top_k)) < dropped] = -1
    if rows > 2:
        ids[1] = -1  # a token without experts
    row = ref.sort_slots(ids, E)[1].reshape(rows, top_k)
    return row, g.random((rows, top_k)).astype(np.float32)


SHAPES = [(1, 1, 8), (1, 8, 7168), (6, 1, 520), (9, 1, 4096), (3, 1, 2056), (7, 3, 264), (5, 4, 2048), (600, 5, 512), (3, 2, 136), (50, 8, 2048), (17, 13, 4104), (9, 64, 256), (2, 4, 20000)]


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,top_k,N", SHAPES)
def test_combine(rows, top_k, N, weighted, residual):
    row, w = _routed(rows, top_k, 8, seed=N)
    n = rows * top_k
    C = _rand((n, N), torch.bfloat16, seed=1, spread=1.0)
    live = np.zeros(n, bool)
    live[row[row >= 0]] = True
    C[torch.from_numpy(~live)] = float("nan")  # rows of dropped slots are not read
    r = _rand((rows, N), torch.bfloat16, seed=2, spread=1.0) if residual else None
    out = torch.full((rows + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    bsfp8.bsmx_moe_combine(C.cuda(), torch.from_numpy(row).cuda(), out, rows, n, top_k, N,
                           weights=torch.from_numpy(w).cuda() if weighted else None,
                           residual=None if r is None else r.cuda())
    _no_error()
    want, mag = ref.combine(C.double().numpy(), row, w.astype(np.float64) if weighted else None,
                            None if r is None else r.double().numpy())
    got = out[:rows].cpu().double().numpy()
    assert np.all(np.abs(got - want) <= HALF_BF16 * np.abs(want) + (top_k + 1) * 2.0 ** -24 * mag * 1.01)
    assert torch.all(out[rows] == 7.0)


def test_combine_into_the_residual():
    rows, top_k, N = 20, 4, 512
    row, w = _routed(rows, top_k, 8, seed=5)
    C = _rand((rows * top_k, N), torch.bfloat16, seed=1).cuda()
    r = _rand((rows, N), torch.bfloat16, seed=2).cuda()
    out = torch.empty_like(r)
    args = dict(weights=torch.from_numpy(w).cuda())
    bsfp8.bsmx_moe_combine(C, torch.from_numpy(row).cuda(), out, rows, rows * top_k, top_k, N, residual=r, **args)
    bsfp8.bsmx_moe_combine(C, torch.from_numpy(row).cuda(), r, rows, rows * top_k, top_k, N, residual=r, **args)
    assert torch.equal(out, r)


@pytest.mark.parametrize("rows,top_k,N", SHAPES)
def test_combine_backward(rows, top_k, N):
    row, w = _routed(rows, top_k, 8, seed=N + 1)
    n = rows * top_k
    C = _rand((n, N), torch.bfloat16, seed=1, spread=1.0)
    named = np.zeros(n, bool)
    named[row[row >= 0]] = True
    C[torch.from_numpy(~named)] = float("nan")
    d = _rand((rows, N), torch.bfloat16, seed=2, spread=1.0)
    dC = torch.full((n + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((n + 3,), 7.0, device="cuda")
    args = (d.cuda(), C.cuda(), torch.from_numpy(row).cuda(), torch.from_numpy(w).cuda())
    bsfp8.bsmx_moe_combine_backward(*args, dC, dw, rows, n, top_k, N)
    _no_error()
    want_C, want_w, mag = ref.combine_backward(d.double().numpy(), C.double().numpy(), row, w.astype(np.float64))
    got = dC[:n].cpu().double().numpy()
    assert np.all(np.abs(got[named] - want_C[named]) <= (HALF_BF16 + 2.0 ** -23) * np.abs(want_C[named]))
    assert np.all(got[~named] == 7.0) and torch.all(dC[n] == 7.0)
    terms = 2 * (8 * -(-N // 2048) + 5 + 8)
    assert np.all(np.abs(dw[:n].view(rows, top_k).cpu().double().numpy() - want_w) <= terms * 2.0 ** -24 * mag)
    assert torch.all(dw[n:] == 7.0)
    again, again_w = torch.full_like(dC, 7.0), torch.full_like(dw, 7.0)
    bsfp8.bsmx_moe_combine_backward(*args, again, again_w, rows, n, top_k, N)
    assert torch.equal(dC, again) and torch.equal(dw, again_w)


def test_combine_backward_against_differences():
    # out is linear in the weights, and a single weight of 1 leaves a row of C unrounded: the
    # difference quotient of <d_out, out> in that weight is exact up to the dot product's order
    rows, top_k, N = 12, 3, 1024
    row, w = _routed(rows, top_k, 4, seed=8, dropped=0.1)
    C = _rand((rows * top_k, N), torch.bfloat16, seed=1, spread=0.5).cuda()
    d = _rand((rows, N), torch.bfloat16, seed=2, spread=0.5).cuda()
    rd = torch.from_numpy(row).cuda()
    dC, dw = torch.zeros_like(C), torch.empty(rows, top_k, device="cuda")
    bsfp8.bsmx_moe_combine_backward(d, C, rd, torch.from_numpy(w).cuda(), dC, dw, rows, rows * top_k, top_k, N)
    for j in range(top_k):
        one = torch.zeros(rows, top_k, device="cuda")
        one[:, j] = 1
        out = torch.empty_like(d)
        bsfp8.bsmx_moe_combine(C, rd, out, rows, rows * top_k, top_k, N, weights=one)
        p = d.double() * out.double()
        assert torch.all((p.sum(1) - dw[:, j].double()).abs() <= 50 * 2.0 ** -24 * p.abs().sum(1))
    # and in a row of C: a change of that row by its own power of two moves <d_out, out> by
    # weight * <d_out, change>
    live = torch.from_numpy(row >= 0)
    t, j = [int(v) for v in torch.nonzero(live)[0]]
    delta = torch.zeros(N, dtype=torch.float64, device="cuda")
    delta[::3] = 1.0
    want = float((dC[row[t, j]].double() * delta).sum())
    exact = float(w[t, j]) * float((d[t].double() * delta).sum())
    assert abs(want - exact) <= HALF_BF16 * float(w[t, j]) * float((d[t].double() * delta).abs().sum())


def test_combine_backward_of_rows_against_differences():
    # weights that are powers of two leave w * C, one row at a time, unrounded: the change of
    # <d_out, out> as a row goes from 0 to a change is exact, and so is dC
    rows, top_k, N = 5, 2, 256
    row = torch.arange(rows * top_k, dtype=torch.int32, device="cuda").flip(0).contiguous()
    w = torch.tensor([0.5, 2.0], device="cuda").repeat(rows, 1)
    d = _rand((rows, N), torch.bfloat16, seed=2, spread=0.5).cuda()
    change = _rand((rows * top_k, N), torch.bfloat16, seed=3, spread=0.5).cuda()
    dC, dw = torch.zeros_like(change), torch.empty(rows, top_k, device="cuda")
    bsfp8.bsmx_moe_combine_backward(d, change, row, w, dC, dw, rows, rows * top_k, top_k, N)
    for r in range(rows * top_k):
        C, out = torch.zeros_like(change), torch.empty_like(d)
        C[r] = change[r]
        bsfp8.bsmx_moe_combine(C, row, out, rows, rows * top_k, top_k, N, weights=w)
        moved = (d.double() * out.double()).sum()
        assert moved == (dC[r].double() * change[r].double()).sum()


def test_dispatch_gradient_is_the_unweighted_combine():
    rows, top_k, K = 30, 4, 384
    row, _ = _routed(rows, top_k, 8, seed=3)
    dA = _rand((rows * top_k, K), torch.bfloat16, seed=7, spread=0.3)
    dx = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    bsfp8.bsmx_moe_combine(dA.cuda(), torch.from_numpy(row).cuda(), dx, rows, rows * top_k, top_k, K)
    x = np.zeros((rows, K))
    for t in range(rows):
        for j in range(top_k):
            if row[t, j] >= 0:
                x[t] += dA[row[t, j]].double().numpy()
    assert np.all(np.abs(dx.cpu().double().numpy() - x) <= HALF_BF16 * np.abs(x) + 1e-5)


# ------------------------------------------------------------------------------ refusals
def test_binding_refuses_wrong_tensors():
    T, K = 4, 256
    bf = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, s = _operand("mxfp8", T, K)
    ids = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, 2, device="cuda")
    for bad in (lambda: bsfp8.bsmx_quantize("mxfp8", bf(K, T).t(), q, s, T, K),
                lambda: bsfp8.bsmx_quantize("mxfp8", bf(T, K).cpu(), q, s, T, K),
                lambda: bsfp8.bsmx_quantize("mxfp8", bf(T - 1, K), q, s, T, K),
                lambda: bsfp8.bsmx_quantize("mxfp8", bf(T, K).double(), q, s, T, K),
                lambda: bsfp8.bsmx_quantize("mxfp8", bf(T, K), q[: T * K - 1], s, T, K),
                lambda: bsfp8.bsmx_quantize("mxfp8", bf(T, K), q, s[: T * K // 32 - 1], T, K),
                lambda: bsfp8.bsmx_quantize("blockwise", bf(T, K), q, s, T, K),
                lambda: bsfp8.bsmx_quantize("mxfp8", bf(T, K), q, s, T, K, x_type="fp32"),
                lambda: bsfp8.bsmx_quantize("mxfp8", bf(T, K), q, s, T, K, row_of_slot=ids.long(), top_k=2, out_rows=8),
                lambda: bsfp8.bsmx_quantize("mxfp8", bf(T, K), q, s, T, K, row_of_slot=ids, top_k=2, out_rows=8),
                lambda: bsfp8.bsmx_rmsnorm_quant("mxfp8", bf(T, K), bf(K - 1), 1e-6, T, K, y=bf(T, K)),
                lambda: bsfp8.bsmx_rmsnorm_quant("mxfp8", bf(T, K), bf(K).float(), 1e-6, T, K, y=bf(T, K)),
                lambda: bsfp8.bsmx_rmsnorm_quant("mxfp8", bf(T, K), bf(K), 1e-6, T, K, residual=bf(T, K),
                                                 residual_out=bf(T, K).float()),
                lambda: bsfp8.bsmx_swiglu_quant("mxfp8", bf(T, K), q, s, T, K),
                lambda: bsfp8.bsmx_moe_sort(ids, ids.reshape(-1)[:5], ids, None, T, 2, 8),
                lambda: bsfp8.bsmx_moe_combine(bf(8, K), ids, bf(T, K), T, 9, 2, K, weights=w),
                lambda: bsfp8.bsmx_moe_combine(bf(8, K), ids, bf(T, K), T, 8, 2, K, weights=w.to(torch.bfloat16)),
                lambda: bsfp8.bsmx_moe_combine_backward(bf(T, K), bf(8, K), ids, w, bf(8, K), w[:3], T, 8, 2, K)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bsfp8.BsFp8Error):
        bsfp8.bsmx_moe_sort(torch.zeros(50000, 2, dtype=torch.int32, device="cuda"), torch.zeros(10, dtype=torch.int32, device="cuda"),
                            torch.zeros(100000, dtype=torch.int32, device="cuda"), None, 50000, 2, 8)
    _no_error()


# ------------------------------------------------------------- streams, graphs, empty, large
def test_chain_of_small_calls_back_to_back():
    # each small kernel may start before the one before it ends: the chain's values show whether
    # each waited for it
    rows, K, top_k, E = 24, 2048, 4, 8
    g = np.random.default_rng(1)
    ids = torch.from_numpy(g.integers(0, E, size=(rows, top_k)).astype(np.int32)).cuda()
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    half = torch.full((rows, top_k), 0.25, device="cuda")
    n = rows * top_k
    ones = torch.ones(n, K, dtype=torch.bfloat16, device="cuda")
    row, off = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(E + 2, dtype=torch.int32, device="cuda")

    def chain(x, steps, sync):
        for _ in range(steps):
            y, C = torch.empty_like(x), torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")
            q, s = _operand("mxfp8", rows, K)
            dw = torch.empty(rows, top_k, device="cuda")
            out = torch.empty_like(x)
            for call in (lambda: bsfp8.bsmx_rmsnorm_quant("mxfp8", x, w, 1e-6, rows, K, y=y),
                         lambda: bsfp8.bsmx_moe_sort(ids, off, row, None, rows, top_k, E),
                         lambda: bsfp8.bsmx_moe_combine_backward(y, ones, row, half, C, dw, rows, n, top_k, K),
                         lambda: bsfp8.bsmx_moe_combine(C, row, out, rows, n, top_k, K),
                         lambda: bsfp8.bsmx_quantize("mxfp8", out, q, s, rows, K)):
                call()
                if sync:
                    torch.cuda.synchronize()
            x = out
        return x, q, s

    x = _rand((rows, K), torch.bfloat16, seed=4, spread=0.5).cuda()
    for a, b in zip(chain(x, 12, False), chain(x, 12, True)):
        assert torch.equal(a, b)


def test_empty_calls():
    bsfp8.bsmx_quantize("mxfp8", None, None, None, 0, 256, x_type="bf16")
    bsfp8.bsmx_swiglu_quant("mxfp8", None, None, None, 0, 256)
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    bsfp8.bsmx_rmsnorm_quant("mxfp8", None, w, 1e-6, 0, 256)
    bsfp8.bsmx_moe_combine(None, None, None, 0, 0, 2, 256)
    bsfp8.bsmx_moe_combine_backward(None, None, None, None, None, None, 0, 0, 2, 256)
    _no_error()


def test_on_another_stream_and_in_a_graph():
    rows, K, top_k, E = 64, 1024, 4, 16
    g = np.random.default_rng(0)
    ids = torch.from_numpy(g.integers(-1, E, size=(rows, top_k)).astype(np.int32)).cuda()
    x = _rand((rows, K), torch.bfloat16, seed=1).cuda()
    n = rows * top_k
    bufs = lambda: dict(off=torch.zeros(E + 2, dtype=torch.int32, device="cuda"),  # noqa: E731
                        row=torch.zeros(n, dtype=torch.int32, device="cuda"),
                        q=torch.zeros(n, K, dtype=torch.uint8, device="cuda"),
                        s=torch.zeros(n, K // 32, dtype=torch.uint8, device="cuda"))

    def go(b, stream=None):
        bsfp8.bsmx_moe_sort(ids, b["off"], b["row"], None, rows, top_k, E, stream=stream)
        bsfp8.bsmx_quantize("mxfp8", x, b["q"], b["s"], rows, K, row_of_slot=b["row"], top_k=top_k, out_rows=n, stream=stream)

    base, other, graphed = bufs(), bufs(), bufs()
    go(base)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    go(other, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(graphed)
    graph.replay()
    torch.cuda.synchronize()
    for k in base:
        assert torch.equal(base[k], other[k]) and torch.equal(base[k], graphed[k])


def test_offsets_past_32_bits():
    # operands of more than 2^31 elements: the last rows are right
    rows, K = 300_001, 7168
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    tail = _rand((4, K), torch.bfloat16, seed=6, spread=0.5)
    x[-4:] = tail.cuda()
    q = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, K // 32, dtype=torch.uint8, device="cuda")
    bsfp8.bsmx_quantize("mxfp8", x, q, s, rows, K)
    ref.check_quantised(tail.double().numpy(), q[-4:], s[-4:], "mxfp8", 0.0, 0.0)
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    bsfp8.bsmx_rmsnorm_quant("mxfp8", x, w, 1e-6, rows, K, residual=x, residual_out=x)
    assert torch.equal(x[-4:].cpu(), (tail.float() * 2).to(torch.bfloat16))
    x[-4:] = tail.cuda()
    row = torch.tensor([[rows - 2, rows - 1]], dtype=torch.int32, device="cuda")
    out = torch.empty(1, K, dtype=torch.bfloat16, device="cuda")
    bsfp8.bsmx_moe_combine(x, row, out, 1, rows, 2, K)
    want = tail[-2].float() + tail[-1].float()
    assert torch.equal(out[0].cpu(), want.to(torch.bfloat16))
    h = x.view(-1)[: (rows // 2) * 2 * K].view(rows // 2, 2 * K)
    h[-1] = _rand((1, 2 * K), torch.bfloat16, seed=3, spread=0.0).cuda()[0]
    bsfp8.bsmx_swiglu_quant("mxfp8", h, q, s, rows // 2, K)
    q2, s2 = torch.empty(1, K, dtype=torch.uint8, device="cuda"), torch.empty(1, K // 32, dtype=torch.uint8, device="cuda")
    bsfp8.bsmx_swiglu_quant("mxfp8", h[-1:].clone(), q2, s2, 1, K)
    assert torch.equal(q.view(-1, K)[rows // 2 - 1], q2[0]) and torch.equal(s.view(-1, K // 32)[rows // 2 - 1], s2[0])
    _no_error()


def test_mapped_rows_and_gradient_past_32_bits():
    rows, K = 300_001, 7168  # of q, C and dC: more than 2^31 elements
    place = torch.tensor([[rows - 1, 0], [rows - 3, -1]], dtype=torch.int32, device="cuda")
    x = _rand((2, K), torch.bfloat16, seed=6, spread=0.5).cuda()
    for fmt in ("mxfp8", "blockwise"):
        want_q, want_s = _operand(fmt, 2, K)
        bsfp8.bsmx_quantize(fmt, x, want_q, want_s, 2, K)
        q = torch.zeros(rows, K, dtype=torch.uint8, device="cuda")
        s = torch.zeros(K // 128, rows, device="cuda") if fmt == "blockwise" else torch.zeros(rows, K // 32, dtype=torch.uint8, device="cuda")
        bsfp8.bsmx_quantize(fmt, x, q, s, 2, K, row_of_slot=place, top_k=2, out_rows=rows)
        _no_error()
        want_q = want_q[: 2 * K].view(2, K)
        want_s = want_s[: K // 64].view(-1, 2).t() if fmt == "blockwise" else want_s[: K // 16].view(2, -1)
        for row, t in ((rows - 1, 0), (0, 0), (rows - 3, 1)):
            assert torch.equal(q[row], want_q[t]) and torch.equal(s[:, row] if fmt == "blockwise" else s[row], want_s[t])
        assert not q[1: rows - 3].any() and not q[rows - 2].any()
        del q, s
    C = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    C[-1], C[-3], C[0] = x[0], x[1], 1
    dC, w = torch.zeros_like(C), torch.tensor([[0.5, 2.0], [4.0, 1.0]], device="cuda")
    d = _rand((2, K), torch.bfloat16, seed=7, spread=0.0).cuda()
    dw = torch.empty(2, 2, device="cuda")
    bsfp8.bsmx_moe_combine_backward(d, C, place, w, dC, dw, 2, rows, 2, K)
    _no_error()
    # weights that are powers of two leave the products unrounded
    assert torch.equal(dC[-1], d[0] * 0.5) and torch.equal(dC[0], d[0] * 2) and torch.equal(dC[-3], d[1] * 4)
    assert not dC[1: rows - 3].any() and not dC[-2].any()
    want, mag = torch.zeros(2, 2, dtype=torch.float64), torch.zeros(2, 2, dtype=torch.float64)
    for t, j, v in ((0, 0, x[0]), (0, 1, torch.ones_like(x[0])), (1, 0, x[1])):
        p = (d[t].double() * v.double()).cpu()
        want[t, j], mag[t, j] = p.sum(), p.abs().sum()
    terms = 2 * (8 * -(-K // 2048) + 5 + 8)
    assert torch.all((dw.cpu().double() - want).abs() <= terms * 2.0 ** -24 * mag)


def test_sort_of_almost_2_to_the_31_slots():
    rows, top_k, E = (1 << 25) - 1, 64, 64
    n = rows * top_k
    ids = torch.arange(64, dtype=torch.int32, device="cuda").repeat(rows)  # slot s goes to expert s % 64
    off = torch.empty(E + 2, dtype=torch.int32, device="cuda")
    row, slot = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(bsfp8.bsmx_moe_sort_workspace(rows, top_k, E), dtype=torch.uint8, device="cuda")
    bsfp8.bsmx_moe_sort(ids, off, row, ws, rows, top_k, E, slot_of_row=slot)
    assert off.tolist() == [e * rows for e in range(E + 1)] + [n]
    e = torch.arange(64, device="cuda")
    for t0 in range(0, rows, 1 << 22):
        t = torch.arange(t0, min(t0 + (1 << 22), rows), device="cuda")
        assert torch.equal(row.view(rows, 64)[t0: t0 + len(t)].long(), e * rows + t[:, None])
        assert torch.equal(slot.view(64, rows)[:, t0: t0 + len(t)].long(), t * 64 + e[:, None])


# ---------------------------------------------------------------------- with the products
def _bf16_bound(want, terms):
    """2 bf16 ulp and 1e-6 of the sum of magnitudes: the grouped GEMM's own bound."""
    e = np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126)))
    return 2 * 2.0 ** (e - 7) + 1e-6 * terms


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantised_rows_are_the_products_operand(fmt):
    m, N, K, E = 9, 256, 1024, 3
    x = _rand((E * m, K), torch.bfloat16, seed=1, spread=0.3)
    W = _rand((E * N, K), torch.float32, seed=2, spread=0.0)
    if fmt == "nvfp4":
        W *= 4
    xq, xs = _operand(fmt, E * m, K)
    bsfp8.bsmx_quantize(fmt, x.cuda(), xq, xs, E * m, K)
    off = torch.arange(0, E * m + 1, m, dtype=torch.int32, device="cuda")
    C = torch.empty(E * m, N, dtype=torch.bfloat16, device="cuda")
    if fmt == "blockwise":  # its weights have 128 x 128 blocks: a scale of 1 here
        wq = (W.clamp(-4, 4)).to(torch.float8_e4m3fn)
        Wd = wq.double().numpy().reshape(E, N, K)
        ws = torch.ones(E, N // 128, K // 128, device="cuda")
        bsfp8.bsfp8_grouped_gemm(xq, wq.cuda().view(torch.uint8), xs, ws, off, C, E * m, N, K, E)
    else:
        wq, ws = _operand(fmt, E * N, K)
        bsfp8.bsmx_quantize(fmt, W.cuda(), wq, ws, E * N, K)
        n = E * N * K
        wv, wsc = ref.decode(wq[: n // (2 if "fp4" in fmt else 1)], ws[: n // ref.VEC[fmt]], fmt, E * N, K)
        Wd = (wv * np.repeat(wsc, ref.VEC[fmt], 1)).reshape(E, N, K)
        bsfp8.bsmx_grouped_gemm(fmt, fmt, xq, wq, xs, ws, off, C, E * m, N, K, E, E)
    _no_error()
    n = E * m * K
    xv, xsc = ref.decode(xq[: n // (2 if "fp4" in fmt else 1)], xs[: n // ref.VEC[fmt]], fmt, E * m, K)
    xd = (xv * np.repeat(xsc, ref.VEC[fmt], 1)).reshape(E, m, K)
    want = np.einsum("emk,enk->emn", xd, Wd).reshape(E * m, N)
    mag = np.einsum("emk,enk->emn", np.abs(xd), np.abs(Wd)).reshape(E * m, N)
    assert np.all(np.abs(C.cpu().double().numpy() - want) <= _bf16_bound(want, mag))
    # and the whole is near the unrounded product
    full = np.einsum("emk,enk->emn", x.double().numpy().reshape(E, m, K), W.double().numpy().reshape(E, N, K)).reshape(E * m, N)
    rel = np.linalg.norm(want - full) / np.linalg.norm(full)
    assert rel < (0.25 if "fp4" in fmt else 0.1)
