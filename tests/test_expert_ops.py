"""The experts' products in 16 bits and the backward pass of the experts on the GPU against their
64-bit definitions (expert_reference.py).

Tolerances, from the arithmetic and set before the first run.  T is the sum of the terms'
magnitudes, and a value's own rounding is at most half a step of its type:
  products   the terms are exact in fp32; every MMA (16 of K, or 32 of 8 bits) and every chunk that
             is added up may lose one unit of the sum, 2^-23 T: (K / 16 + 2) * 2^-23 T
  8 bits     two more roundings of the scales' products
  add        one more rounding in fp32, of a sum that |add| + T bounds
  quantised  the reciprocal and the product, 2^-22, as for the quantisation along the rows
  SwiGLU     (10 + |g|) * 2^-22 of the terms' magnitude: the exponential's argument is rounded to
             2^-24 |g| log2(e), 1 - s to 2^-25 beside g
"""
import threading

import numpy as np
import pytest
import torch

import block_scaled_fp8_persistent_gb300 as bsfp8
import expert_reference as ref
import moe_reference

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
OFFSETS_ERROR, IDS_ERROR, ROWS_ERROR = 6, 8, 11


def _no_error():
    assert bsfp8.bsfp8_get_device_error() == 0


def _rand(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def _close(got, want, tol, dtype):
    """Within tol and the rounding to dtype; nothing but numbers where numbers are due."""
    got = got.double().cpu()
    limit = tol + (want.abs() + tol) * ref.HALF[dtype] + ref.TINY[dtype]
    off = (got - want).abs()
    bad = ~(off <= limit)
    assert not bad.any(), (int(bad.sum()), bad.numel(), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def _guarded(shape, dtype, fill=7.0, offset=0):
    """A buffer of `shape` with 256 guard elements behind it, and all of its memory."""
    n = int(np.prod(shape))
    whole = torch.full((offset + n + 256,), fill, dtype=dtype, device="cuda")
    return whole[offset: offset + n].view(shape), whole


# ------------------------------------------------------------------------------ products
def _product(sizes, N, K, dtype=BF16, transposed=False, ids=None, experts=None, spare=0, seed=0, offset=0, A=None, B=None):
    off = ref.offsets_of(sizes)
    rows = int(off[-1]) + spare
    E = experts or len(sizes)
    A = _rand(seed + 1, rows, K, dtype=dtype) if A is None else A
    B = _rand(seed + 2, *((E, K, N) if transposed else (E, N, K)), dtype=dtype, scale=K ** -0.5) if B is None else B
    C, whole = _guarded((rows, N), dtype, offset=offset)
    bsfp8.bs16_grouped_gemm(A.cuda(), B.cuda(), off.cuda(), C, rows, N, K, len(sizes), E,
                            expert_ids=None if ids is None else torch.tensor(ids, dtype=torch.int32).cuda(), transposed=transposed)
    _no_error()
    kept = int(off[-1])
    assert torch.all(whole[offset + kept * N:] == 7) and torch.all(whole[:offset] == 7)
    want, T = ref.product(A, B, off, ids, transposed)
    _close(C[:kept], want, T * (K / 16 + 2) * 2.0 ** -23, dtype)


SIZES = [[1], [0, 2, 0], [33, 0, 31, 1], [5, 32, 27], [100, 28, 0, 129], [128], [129, 127], [300, 0, 513, 1], [255, 257, 256]]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("N,K", [(128, 64), (264, 200), (8, 8)])
def test_product(sizes, N, K, transposed, dtype):
    _product(sizes, N, K, dtype, transposed, seed=N + K)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes", [[3, 2], [70, 30], [300, 200]], ids=str)
@pytest.mark.parametrize("N,K", [(16, 72), (24, 1032), (120, 56), (136, 128), (248, 136), (520, 16), (1000, 520), (512, 7168)])
def test_product_odd_sides(sizes, N, K, transposed):
    _product(sizes, N, K, BF16, transposed, seed=N)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes,N,K", [
    ([1], 128, 256), ([1], 128, 512), ([3, 2], 136, 1024), ([1], 2048, 1024), ([20, 12, 32], 256, 1032),  # K shared by 2, 4, 8
    ([65, 500], 264, 640), ([100], 1024, 4096), ([700], 520, 1024),  # tiles of 64 rows
    ([1300, 1200], 1536, 136), ([2600], 1600, 72),  # of 128
    ([2500, 2440], 2048, 72), ([2000, 1, 3000], 2568, 136),  # of 256
    ([520, 1000, 3, 255, 256, 257, 511, 513, 0, 2500, 700, 900], 17416, 72),  # of 512
], ids=str)
def test_product_every_tile(sizes, N, K, transposed):
    _product(sizes, N, K, BF16, transposed, seed=3)


@pytest.mark.parametrize("sizes", [[9, 0, 20], [90, 0, 100], [300, 0, 280]], ids=str)
def test_product_behind_the_last_group(sizes):
    _product(sizes, 136, 264, spare=40)


@pytest.mark.parametrize("sizes", [[9, 3, 0, 20], [290, 130, 0, 200]], ids=str)
@pytest.mark.parametrize("transposed", [False, True])
def test_product_expert_ids(sizes, transposed):
    _product(sizes, 264, 136, transposed=transposed, ids=[4, 1, 0, 4], experts=5)


@pytest.mark.parametrize("sizes", [[9, 3], [90, 40], [290, 130]], ids=str)
def test_product_output_aligned_to_16_bytes_only(sizes):
    _product(sizes, 272, 64, offset=8)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes", [[9, 0, 3], [90, 0, 40], [290, 0, 130]], ids=str)
def test_product_other_groups_do_not_reach_a_row(sizes, transposed):
    # NaN in the rows of the second and third group and in all weights but the first's
    N, K = 200, 72
    off = ref.offsets_of(sizes)
    rows = int(off[-1])
    A = _rand(1, rows, K)
    A[sizes[0]:] = float("nan")
    B = _rand(2, *((3, K, N) if transposed else (3, N, K)))
    B[1:] = float("nan")
    C = torch.zeros(rows, N, dtype=BF16, device="cuda")
    bsfp8.bs16_grouped_gemm(A.cuda(), B.cuda(), off.cuda(), C, rows, N, K, 3, 3, transposed=transposed)
    _no_error()
    want, T = ref.product(A[: sizes[0]], B, ref.offsets_of(sizes[:1]), None, transposed)
    _close(C[: sizes[0]], want, T * (K / 16 + 2) * 2.0 ** -23, BF16)
    assert torch.isnan(C[sizes[0]:]).all()


def test_product_special_values():
    A = torch.ones(3, 64, dtype=FP16)
    A[1] = 60000
    A[2, 5] = float("inf")
    B = torch.ones(1, 16, 64, dtype=FP16)
    B[0, 3] = 0
    C = torch.zeros(3, 16, dtype=FP16, device="cuda")
    bsfp8.bs16_grouped_gemm(A.cuda(), B.cuda(), ref.offsets_of([3]).cuda(), C, 3, 16, 64, 1, 1)
    got = C.cpu()
    assert torch.all(got[0, :3] == 64) and got[0, 3] == 0
    assert torch.isinf(got[1, 0]) and got[1, 3] == 0
    assert torch.isinf(got[2, 0]) and torch.isnan(got[2, 3])


def test_product_many_groups():
    sizes = [(7 * i) % 5 for i in range(300)]
    _product(sizes, 128, 64, seed=5)


# ------------------------------------------------------------------------------ weight gradients
def _add(E, N, K, dtype, seed):
    return _rand(seed, E, N, K, dtype=dtype, scale=3.0)


def _wgrad(sizes, N, K, dtype=BF16, out=None, add=False, spare=0, in_place=False, offset=0):
    off = ref.offsets_of(sizes)
    rows, E, out = int(off[-1]) + spare, len(sizes), out or dtype
    dC, A = _rand(N, rows, N, dtype=dtype), _rand(K + 1, rows, K, dtype=dtype)
    if spare:
        dC[rows - spare:] = float("nan")
        A[rows - spare:] = float("inf")
    dB, whole = _guarded((E, N, K), out, offset=offset)
    plus = _add(E, N, K, out, 5) if add else None
    if in_place:
        dB.copy_(plus)
    bsfp8.bs16_grouped_wgrad(dC.cuda(), A.cuda(), off.cuda(), dB, rows, N, K, E,
                             add=None if plus is None else dB if in_place else plus.cuda())
    _no_error()
    assert torch.all(whole[offset + E * N * K:] == 7) and torch.all(whole[:offset] == 7)
    want, T = ref.wgrad(dC, A, off)
    longest = max(sizes) if sizes else 0
    tol = T * (longest / 16 + 2) * 2.0 ** -23
    if add:
        want = want + plus.double()
        tol = tol + (plus.double().abs() + T) * 2.0 ** -24
    _close(dB, want, tol, out)


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, FP32), (FP16, FP16), (FP16, FP32)])
@pytest.mark.parametrize("sizes", SIZES + [[63, 64, 65, 0, 16, 17], [1000, 513]], ids=str)
@pytest.mark.parametrize("N,K", [(128, 64), (264, 200)])
def test_wgrad(sizes, N, K, dtype, out):
    _wgrad(sizes, N, K, dtype, out)


@pytest.mark.parametrize("N,K", [(8, 8), (16, 136), (136, 24), (120, 264), (520, 1032), (256, 256)])
def test_wgrad_odd_sides(N, K):
    _wgrad([70, 3, 0, 130], N, K)


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, FP32), (FP16, FP16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_wgrad_added(dtype, out, in_place):
    _wgrad([70, 0, 130], 136, 264, dtype, out, add=True, in_place=in_place)


@pytest.mark.parametrize("sizes", [[70, 0, 130], [128, 64], [1], [0, 0]], ids=str)
def test_wgrad_rows_behind_the_last_group(sizes):
    _wgrad(sizes, 136, 264, spare=90)


# few tiles and many rows: the rows of a tile are shared by several pairs of SMs
MANY_ROWS = [[1024], [1025], [1400], [4097], [2900, 3, 0, 1300], [0, 2100], [9000]]


@pytest.mark.parametrize("dtype,out,add", [(BF16, FP32, False), (FP16, FP16, True), (BF16, BF16, False), (BF16, FP32, True)])
@pytest.mark.parametrize("sizes", MANY_ROWS, ids=str)
def test_wgrad_many_rows_few_tiles(sizes, dtype, out, add):
    _wgrad(sizes, 264, 136, dtype, out, add=add, spare=33)


@pytest.mark.parametrize("offset", [8, 16])
def test_wgrad_output_alignment(offset):
    _wgrad([70, 30], 136, 264, BF16, FP32, add=True, in_place=True, offset=offset // 2)


def test_wgrad_other_groups_do_not_reach_the_sum():
    for bad in (float("nan"), float("inf")):
        sizes, N, K = [37, 90, 5], 136, 136
        off = ref.offsets_of(sizes)
        dC, A = _rand(1, 132, N), _rand(2, 132, K)
        dC[37:127], A[37:127] = bad, bad
        dB = torch.zeros(3, N, K, dtype=FP32, device="cuda")
        bsfp8.bs16_grouped_wgrad(dC.cuda(), A.cuda(), off.cuda(), dB, 132, N, K, 3)
        want, T = ref.wgrad(dC, A, off)
        for e in (0, 2):
            _close(dB[e], want[e], T[e] * 10 * 2.0 ** -23, FP32)
        assert torch.equal(torch.isnan(dB[1].cpu()), torch.isnan(want[1]))


def test_wgrad_without_rows():
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    plus = _add(3, 64, 128, FP32, 1).cuda()
    dB = torch.full((3, 64, 128), 7.0, device="cuda")
    bsfp8.bs16_grouped_wgrad(None, None, off, dB, 0, 64, 128, 3, type="bf16")
    assert torch.all(dB == 0)
    bsfp8.bs16_grouped_wgrad(None, None, off, dB, 0, 64, 128, 3, type="fp16", add=plus)
    assert torch.equal(dB, plus)
    _no_error()


# ------------------------------------------------------------------------------ 8-bit gradients
def _wgrad8(sizes, N, K, out=FP32, add=False, spare=0, in_place=False):
    off = ref.offsets_of(sizes)
    rows, E = int(off[-1]) + spare, len(sizes)
    spread = torch.exp(torch.randn(1, N, generator=torch.Generator().manual_seed(3)))
    dC, sc = ref.quantise_columns(_rand(N, rows, N, dtype=FP32) * spread, off)
    A, sa = ref.quantise_columns(_rand(K + 1, rows, K, dtype=FP32), off)
    dC[rows - spare:] = 0x7F  # NaN
    A[rows - spare:] = 0x7F
    used = torch.zeros(sc.shape[0], dtype=torch.bool)
    used[[s for s, _, _ in ref.blocks_of(off)]] = True
    sc[~used], sa[~used] = float("nan"), float("nan")
    dB, whole = _guarded((E, N, K), out)
    plus = _add(E, N, K, out, 5) if add else None
    if in_place:
        dB.copy_(plus)
    bsfp8.bsfp8_grouped_wgrad(dC.cuda(), A.cuda(), sc.cuda(), sa.cuda(), off.cuda(), dB, rows, N, K, E,
                              add=None if plus is None else dB if in_place else plus.cuda())
    _no_error()
    assert torch.all(whole[E * N * K:] == 7)
    want, T = ref.wgrad(ref.dequantised_columns(dC, sc, off), ref.dequantised_columns(A, sa, off), off)
    tol = T * (max(sizes) / 32 + 6) * 2.0 ** -23
    if add:
        want = want + plus.double()
        tol = tol + (plus.double().abs() + T) * 2.0 ** -24
    _close(dB, want, tol, out)


@pytest.mark.parametrize("out", [FP32, BF16, FP16])
@pytest.mark.parametrize("sizes", SIZES + [[31, 32, 33, 0, 127], [1000, 513, 0, 384]], ids=str)
@pytest.mark.parametrize("N,K", [(128, 128), (384, 640)])
def test_wgrad8(sizes, N, K, out):
    _wgrad8(sizes, N, K, out)


@pytest.mark.parametrize("out,add", [(FP32, False), (FP16, True), (BF16, False), (FP32, True)])
@pytest.mark.parametrize("sizes", MANY_ROWS, ids=str)
def test_wgrad8_many_rows_few_tiles(sizes, out, add):
    _wgrad8(sizes, 384, 128, out, add=add, spare=33)


@pytest.mark.parametrize("out", [FP32, BF16])
@pytest.mark.parametrize("in_place", [False, True])
def test_wgrad8_added(out, in_place):
    _wgrad8([70, 0, 130, 300], 256, 384, out, add=True, in_place=in_place)


@pytest.mark.parametrize("sizes", [[70, 0, 130], [128, 256], [1], [0, 0]], ids=str)
def test_wgrad8_rows_behind_the_last_group(sizes):
    _wgrad8(sizes, 256, 128, spare=90)


def test_wgrad8_exact_values():
    # small integers under powers of two: every sum is exact, so the results are equal
    sizes, N, K = [200, 57, 0, 129], 256, 384
    off = ref.offsets_of(sizes)
    g = torch.Generator().manual_seed(1)
    dC, A = (torch.randint(-3, 4, (386, n), generator=g).float().to(ref.E4M3).view(torch.uint8) for n in (N, K))
    blocks = 386 // 128 + 4
    sc, sa = (torch.exp2(torch.randint(-3, 4, (blocks, n), generator=g).float()) for n in (N, K))
    dB = torch.zeros(4, N, K, device="cuda")
    bsfp8.bsfp8_grouped_wgrad(dC.cuda(), A.cuda(), sc.cuda(), sa.cuda(), off.cuda(), dB, 386, N, K, 4)
    want, _ = ref.wgrad(ref.dequantised_columns(dC, sc, off), ref.dequantised_columns(A, sa, off), off)
    assert torch.equal(dB.double().cpu(), want)


def test_wgrad8_nan_scale_spoils_its_column_only():
    sizes, N, K = [200, 100], 128, 256
    off = ref.offsets_of(sizes)
    x = _rand(1, 300, N, dtype=FP32)
    dC, sc = ref.quantise_columns(x, off)
    A, sa = ref.quantise_columns(_rand(2, 300, K, dtype=FP32), off)
    sc[1, 5] = float("nan")  # the second block of group 0
    dB = torch.zeros(2, N, K, device="cuda")
    bsfp8.bsfp8_grouped_wgrad(dC.cuda(), A.cuda(), sc.cuda(), sa.cuda(), off.cuda(), dB, 300, N, K, 2)
    bad = torch.isnan(dB)
    assert bad[0, 5].all() and bad.sum() == K


# ------------------------------------------------------------------------------ columns
def _check_columns(x, off, q, scales, u=2.0 ** -22):
    for s, r0, r1 in ref.blocks_of(off):
        v = np.zeros((x.shape[1], 128))
        v[:, : r1 - r0] = x[r0:r1].double().t().numpy()
        codes = torch.zeros(x.shape[1], 128, dtype=torch.uint8)
        codes[:, : r1 - r0] = q[r0:r1].t()
        moe_reference.check_quantised(v, codes, scales[s].contiguous(), "blockwise", u, u)


def _columns(sizes, K, dtype, spare=0):
    off = ref.offsets_of(sizes)
    rows = int(off[-1]) + spare
    x = _rand(K + rows, rows, K, dtype=FP32)
    x = (x * torch.exp(torch.randn(1, K, generator=torch.Generator().manual_seed(4)))).to(dtype)
    x[:, 3] = 0
    if spare:
        x[rows - spare:] = float("nan")
    q, q_all = _guarded((rows, K), torch.uint8, fill=7)
    s, s_all = _guarded((rows // 128 + len(sizes), K), FP32)
    bsfp8.bsfp8_quantize_columns(x.cuda(), off.cuda(), q, s, rows, K, len(sizes))
    _no_error()
    assert torch.all(q_all[int(off[-1]) * K:] == 7) and torch.all(s_all[s.numel():] == 7)
    used = [b for b, _, _ in ref.blocks_of(off)]
    unused = [b for b in range(s.shape[0]) if b not in used]
    assert torch.all(s[unused] == 7)
    _check_columns(x, off, q.cpu(), s.cpu())


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("sizes", SIZES + [[127, 128, 129, 0, 15, 17], [1000]], ids=str)
def test_columns(sizes, dtype):
    _columns(sizes, 256, dtype)


@pytest.mark.parametrize("K", [128, 384, 7168])
def test_columns_widths(K):
    _columns([70, 0, 130], K, BF16, spare=5)


def test_columns_many_groups():
    _columns([(7 * i) % 5 for i in range(700)], 128, BF16)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_columns_non_finite_blocks_have_nan_scales(bad):
    x = _rand(1, 300, 128)
    x[140, 9] = bad
    off = ref.offsets_of([130, 170])
    q, s = torch.zeros(300, 128, dtype=torch.uint8, device="cuda"), torch.zeros(4, 128, device="cuda")
    bsfp8.bsfp8_quantize_columns(x.cuda(), off.cuda(), q, s, 300, 128, 2)
    nan = torch.isnan(s)
    assert nan[2, 9] and nan.sum() == 1  # block 0 of group 1 has row 130 / 128 + 1 = 2
    _no_error()


@pytest.mark.parametrize("top_k", [1, 3])
def test_columns_gathered(top_k):
    sizes, tokens, K = [70, 0, 130, 41], 100, 256
    rows = tokens * top_k
    off = ref.offsets_of(sizes) if top_k == 3 else ref.offsets_of([40, 0, 30, 20])
    x = _rand(1, tokens, K)
    slot = torch.randperm(rows, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    slot[11] = -1
    slot[int(off[-1]):] = -1
    q = torch.full((rows, K), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((rows // 128 + 4, K), 7.0, device="cuda")
    bsfp8.bsfp8_quantize_columns(x.cuda(), off.cuda(), q, s, rows, K, 4, slot_of_row=slot.cuda(), top_k=top_k)
    _no_error()
    gathered = x[slot.clamp(min=0).long() // top_k].clone()
    gathered[slot < 0] = 0
    _check_columns(gathered, off, q.cpu(), s.cpu())
    assert torch.all(q[int(off[-1]):] == 7)


def test_columns_gathered_out_of_range_is_recorded():
    x, off = _rand(1, 10, 128), ref.offsets_of([10])
    slot = torch.arange(10, dtype=torch.int32)
    slot[4] = 10
    q, s = torch.zeros(10, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, 128, device="cuda")
    bsfp8.bsfp8_quantize_columns(x.cuda(), off.cuda(), q, s, 10, 128, 1, slot_of_row=slot.cuda())
    assert bsfp8.bsfp8_get_device_error() == ROWS_ERROR
    x[4] = 0
    _check_columns(x, off, q.cpu(), s.cpu())


# ------------------------------------------------------------------------------ SwiGLU's gradient
def _gate(seed, rows, N, dtype):
    h = _rand(seed, rows, 2 * N, dtype=FP32, scale=3.0)
    g = h[:, :N]
    near = (g + 1.2785).abs() < 0.2  # d_g crosses zero there: no relative tolerance
    h[:, :N] = torch.where(near, torch.tensor(0.5), g)
    return h.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,N", [(1, 128), (3, 256), (7, 384), (130, 128), (33, 1152), (5, 7168)])
def test_swiglu_backward(rows, N, dtype):
    h, d = _gate(rows, rows, N, dtype), _rand(N, rows, N, dtype=dtype)
    d_h, d_all = _guarded((rows, 2 * N), dtype)
    act, act_all = _guarded((rows, N), dtype)
    bsfp8.bsmx_swiglu_backward(h.cuda(), d.cuda(), rows, N, d_h=d_h, act=act)
    _no_error()
    assert torch.all(d_all[d_h.numel():] == 7) and torch.all(act_all[act.numel():] == 7)
    want_act, want, mag = ref.swiglu_backward(h, d)
    g = h[:, :N].double().abs()
    u = (10 + g) * 2.0 ** -22
    _close(act, want_act, want_act.abs() * u, dtype)
    _close(d_h, want, mag * torch.cat([u, u], dim=1), dtype)
    only = torch.zeros_like(act)
    bsfp8.bsmx_swiglu_backward(h.cuda(), None, rows, N, act=only)
    assert torch.equal(only, act)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4", "blockwise"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("rows,N", [(1, 128), (7, 384), (130, 256)])
def test_swiglu_backward_quantised(rows, N, dtype, fmt):
    h, d = _gate(rows, rows, N, dtype), _rand(N, rows, N, dtype=dtype)
    K = 2 * N
    q = torch.zeros(rows, K // 2 if "fp4" in fmt else K, dtype=torch.uint8, device="cuda")
    shape = (K // 128, rows) if fmt == "blockwise" else (rows, K // moe_reference.VEC[fmt])
    s = torch.zeros(shape, dtype=FP32 if fmt == "blockwise" else torch.uint8, device="cuda")
    bsfp8.bsmx_swiglu_backward(h.cuda(), d.cuda(), rows, N, q=q, scales=s, format=fmt)
    _no_error()
    _, want, mag = ref.swiglu_backward(h, d)
    g = h[:, :N].double().abs()
    u = torch.cat([(10 + g), (10 + g)], dim=1) * 2.0 ** -22
    u = (u * mag / want.abs().clamp(min=1e-300)).numpy()
    u = np.where(want.numpy() == 0, 0, u) + 2.0 ** -22
    moe_reference.check_quantised(want.numpy(), q, s, fmt, u, 2.0 ** -22)


def test_swiglu_backward_extremes():
    g = torch.tensor([0.0, -0.0, 90.0, -90.0, 200.0, -200.0, 3e38, -3e38] * 16).to(BF16)[None]
    h = torch.cat([g, torch.full_like(g, 2.0)], dim=1)
    d = torch.full_like(g, 0.5)
    d_h, act = torch.zeros_like(h).cuda(), torch.zeros_like(g).cuda()
    bsfp8.bsmx_swiglu_backward(h.cuda(), d.cuda(), 1, 128, d_h=d_h, act=act)
    d_g, d_u, act = d_h[0, :8].cpu().float(), d_h[0, 128:136].cpu().float(), act[0, :8].cpu().float()
    assert d_g[0] == 0.5 and d_g[2] == 1 and d_g[4] == 1 and d_g[6] == 1
    assert abs(d_g[3]) < 1e-30 and d_g[5] == 0 and d_g[7] == 0
    assert d_u[0] == 0 and d_u[2] == 45 and abs(d_u[3]) < 1e-30 and d_u[5] == 0
    assert act[0] == 0 and act[2] == 180 and act[5] == 0 and act[7] == 0


def test_swiglu_backward_in_place():
    h, d = _gate(1, 20, 256, BF16).cuda(), _rand(2, 20, 256).cuda()
    d_h, act = torch.empty_like(h), torch.empty_like(d)
    bsfp8.bsmx_swiglu_backward(h, d, 20, 256, d_h=d_h, act=act)
    bsfp8.bsmx_swiglu_backward(h, d, 20, 256, d_h=h, act=d)
    assert torch.equal(h, d_h) and torch.equal(d, act)


def test_swiglu_backward_is_the_derivative():
    # differences of the forward operator in 64 bits
    h, d = _gate(3, 4, 128, BF16), _rand(4, 4, 128)
    d_h = torch.zeros(4, 256, dtype=BF16, device="cuda")
    bsfp8.bsmx_swiglu_backward(h.cuda(), d.cuda(), 4, 128, d_h=d_h)
    x = h.double().requires_grad_()
    gate, up = x.chunk(2, dim=1)
    (gate / (1 + torch.exp(-gate)) * up * d.double()).sum().backward()
    assert torch.allclose(d_h.double().cpu(), x.grad, rtol=2.0 ** -7, atol=1e-6)


# ------------------------------------------------------------------------------ how they are called
def _calls():
    """(outputs, call(stream) of every operator after another, an input)."""
    sizes, N, K = [70, 0, 130, 56], 256, 384
    off = ref.offsets_of(sizes)
    rows = 256
    x, y = _rand(1, rows, N).cuda(), _rand(2, rows, K).cuda()
    W = _rand(3, 4, N, K, scale=0.05).cuda()
    off = off.cuda()
    qx, sx = torch.zeros(rows, N, dtype=torch.uint8, device="cuda"), torch.zeros(6, N, device="cuda")
    qy, sy = torch.zeros(rows, K, dtype=torch.uint8, device="cuda"), torch.zeros(6, K, device="cuda")
    C, dA = torch.zeros(rows, N, dtype=BF16, device="cuda"), torch.zeros(rows, K, dtype=BF16, device="cuda")
    dB, dB8 = torch.zeros(4, N, K, device="cuda"), torch.zeros(4, N, K, device="cuda")
    d_act, d_h = _rand(5, rows, N // 2).cuda(), torch.zeros(rows, N, dtype=BF16, device="cuda")

    def run(stream=None):
        bsfp8.bs16_grouped_gemm(y, W, off, C, rows, N, K, 4, 4, stream=stream)
        bsfp8.bs16_grouped_gemm(C, W, off, dA, rows, K, N, 4, 4, transposed=True, stream=stream)
        bsfp8.bs16_grouped_wgrad(C, dA, off, dB, rows, N, K, 4, stream=stream)
        bsfp8.bsfp8_quantize_columns(C, off, qx, sx, rows, N, 4, stream=stream)
        bsfp8.bsfp8_quantize_columns(dA, off, qy, sy, rows, K, 4, stream=stream)
        bsfp8.bsfp8_grouped_wgrad(qx, qy, sx, sy, off, dB8, rows, N, K, 4, stream=stream)
        bsfp8.bsmx_swiglu_backward(C, d_act, rows, N // 2, d_h=d_h, stream=stream)

    return [C, dA, dB, qx, sx, qy, sy, dB8, d_h], run, y


def test_same_bits_every_time():
    outs, run, _ = _calls()
    run()
    first = [o.clone() for o in outs]
    for o in outs:
        if o.shape[0] != 6:  # (scales that no block has are left as they are)
            o.fill_(3)
    run()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)
    _no_error()


def test_streams_and_graphs():
    outs, run, y = _calls()
    run()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    run(side)
    side.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    keep = y.clone()
    y.copy_(-keep)
    graph.replay()
    y.copy_(keep)
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)
    _no_error()


def test_threads_on_streams_of_their_own():
    sets = [_calls() for _ in range(4)]
    wants = []
    for outs, run, _ in sets:
        run()
        torch.cuda.synchronize()
        wants.append([o.clone() for o in outs])
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(5):
            sets[i][1](s)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for want, (outs, _, _) in zip(wants, sets):
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
    _no_error()


@pytest.mark.parametrize("bad", [[0, 5, 3, 10], [1, 5, 7, 10], [0, 5, 7, 11], [0, -2, 7, 10]], ids=str)
def test_offsets_that_are_no_partition(bad):
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    x, W = _rand(1, 10, 128).cuda(), _rand(2, 3, 128, 128).cuda()
    C = torch.full((10, 128), 7.0, dtype=BF16, device="cuda")
    bsfp8.bs16_grouped_gemm(x, W, off, C, 10, 128, 128, 3, 3)
    assert bsfp8.bsfp8_get_device_error() == OFFSETS_ERROR
    dB = torch.full((3, 128, 128), 7.0, device="cuda")
    bsfp8.bs16_grouped_wgrad(x, x, off, dB, 10, 128, 128, 3)
    assert bsfp8.bsfp8_get_device_error() == OFFSETS_ERROR
    q, s = torch.zeros(10, 128, dtype=torch.uint8, device="cuda"), torch.ones(3, 128, device="cuda")
    bsfp8.bsfp8_grouped_wgrad(q, q, s, s, off, dB, 10, 128, 128, 3)
    assert bsfp8.bsfp8_get_device_error() == OFFSETS_ERROR
    assert torch.all(C == 7) and torch.all(dB == 7)
    bsfp8.bsfp8_quantize_columns(x, off, q, s, 10, 128, 3)
    assert bsfp8.bsfp8_get_device_error() == OFFSETS_ERROR


@pytest.mark.parametrize("ids", [[0, 3], [-1, 0]])
def test_expert_ids_out_of_range(ids):
    x, W = _rand(1, 10, 128).cuda(), _rand(2, 3, 128, 128).cuda()
    C = torch.full((10, 128), 7.0, dtype=BF16, device="cuda")
    bsfp8.bs16_grouped_gemm(x, W, ref.offsets_of([4, 6]).cuda(), C, 10, 128, 128, 2, 3,
                            expert_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))
    assert bsfp8.bsfp8_get_device_error() == IDS_ERROR
    assert torch.all(C == 7)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes", [[0] * 60 + [70, 3], [1] * 40 + [33, 64, 200], [16] * 20 + [600, 0, 5], [31, 1, 0, 0, 0, 0, 0, 40]], ids=str)
@pytest.mark.parametrize("N,K", [(264, 200), (1032, 520)])
def test_product_groups_of_very_different_sizes(sizes, N, K, transposed):
    _product(sizes, N, K, BF16, transposed, seed=N)


@pytest.mark.parametrize("dtype,out", [(BF16, FP32), (FP16, FP16)])
def test_wgrad_many_rows_added_in_place(dtype, out):
    _wgrad([4000, 0, 3001], 264, 200, dtype, out, add=True, in_place=True)


def test_wgrad8_many_rows_added_in_place():
    _wgrad8([4000, 0, 3001], 256, 128, FP32, add=True, in_place=True)


def test_columns_of_no_tokens():
    rows, K = 150, 256
    off, slots = ref.offsets_of([100, 50]).cuda(), torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    q, s = torch.ones(rows, K, dtype=torch.uint8, device="cuda"), torch.zeros(rows // 128 + 2, K, device="cuda")
    bsfp8.bsfp8_quantize_columns(None, off, q, s, rows, K, 2, slot_of_row=slots, top_k=2, x_rows=0, x_type="bf16")
    _no_error()
    assert torch.all(q == 0) and torch.all(s[:2] == 1)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes,N,K", [
    ([49], 816, 2992), ([128], 2048, 1024), ([100], 4096, 520), ([129], 1032, 512), ([40, 0, 77], 1000, 1912),  # K shared by pairs
    ([300], 2048, 1000), ([65, 64, 63, 1], 136, 1032),
], ids=str)
def test_product_tiles_that_share_k(sizes, N, K, transposed):
    _product(sizes, N, K, FP16, transposed, seed=4)


@pytest.mark.parametrize("groups", [191, 192, 193, 400])
@pytest.mark.parametrize("each", [1, 20])
def test_product_as_many_groups_as_are_listed(groups, each):
    # groups with rows between empty ones, under expert ids that go round
    sizes = [each if g % 2 else 0 for g in range(2 * groups)]
    _product(sizes, 72, 136, ids=[g % 5 for g in range(2 * groups)], experts=5)


@pytest.mark.parametrize("groups", [127, 128, 129])
@pytest.mark.parametrize("each,spare", [(1, 0), (40, 3)])
def test_product_about_as_many_groups_as_are_listed(groups, each, spare):
    _product([each if g % 3 else 0 for g in range(groups * 3 // 2)] + [each], 520, 136, spare=spare)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes", [[700, 0, 420, 900, 1], [130] * 24, [2500, 16, 16, 16], [64] * 150], ids=["uneven", "even", "one large", "many"])
@pytest.mark.parametrize("N,K", [(3080, 2048), (3080, 200)])
def test_product_planned_over_several_rounds(sizes, N, K, transposed):
    # more tiles than pairs of SMs, with a plan (K of 32 blocks) and without
    _product(sizes, N, K, BF16, transposed, seed=8)
