"""The experts' operators in the forms that their rules choose for ordinary sizes, and in loops that
are long enough to turn: against 64 bits, with the tolerances of test_expert_ops.py."""
import os
import sys

import pytest
import torch

import block_scaled_fp8_persistent_gb300 as bsfp8
import expert_forms as forms
import expert_reference as ref

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


TYPES = {"bf16": BF16, "fp16": FP16, "fp32": FP32}


def _no_error():
    assert bsfp8.bsfp8_get_device_error() == 0


def _rand(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _groups(sizes):
    off = ref.offsets_of(sizes)
    return off.cuda(), list(enumerate(zip(off.tolist(), off.tolist()[1:])))


def _close(got, want, tol, dtype):
    bad = ~((got.double() - want).abs() <= tol + (want.abs() + tol) * ref.HALF[dtype] + ref.TINY[dtype])
    assert not bad.any(), (int(bad.sum()), bad.numel(), bad.nonzero()[:4].tolist())


# ------------------------------------------------------------------------------ long calls
@pytest.mark.slow
def test_wgrad8_waits_for_a_last_group_behind_a_second_of_whole_stages():
    """1.4 million rows in whole blocks of 128, then 33 more: 2 * 1.4e6 * 2^30 operations take 1.4 s at
    2.1 PFLOP/s, and all of it goes by before the first stage that is not full, while no wait of the
    kernel may last longer than a second without anything happening.  Ones, so that the sums are the
    groups' lengths, exact in fp32."""
    M0, last, N = 10938 * 128, 33, 32768
    rows = M0 + last
    ones = torch.full((rows, N), 0x38, dtype=torch.uint8, device="cuda")  # e4m3 1.0
    scales = torch.ones(rows // 128 + 2, N, device="cuda")
    dB = torch.zeros(2, N, N, device="cuda")
    off = torch.tensor([0, M0, rows], dtype=torch.int32, device="cuda")
    bsfp8.bsfp8_grouped_wgrad(ones, ones, scales, scales, off, dB, rows, N, N, 2)
    _no_error()
    assert torch.all(dB[0] == M0) and torch.all(dB[1] == last)


# ------------------------------------------------------------------------------ long sums
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes,N,K", [
    ([1], 64, 16384), ([1], 64, 131072), ([3, 0, 1], 136, 131080), ([1], 64, 1 << 20),
    ([300], 512, 16384), ([300], 512, 65536), ([300], 512, 65600), ([300], 512, 262144), ([17, 0, 40, 1], 264, 1 << 18), ([300], 264, 1 << 20),
    ([1000, 700, 1, 257], 1032, 16448), ([513, 90], 2048, 40968),
], ids=str)
def test_product_long_sums_of_one_sign(sizes, N, K, transposed, dtype):
    """Terms of one sign, so that what an accumulator loses adds up.  An MMA of 16 loses at most one
    unit of its accumulator's sum, 2^-23 T, and no accumulator takes more than 16384 of K for fp16
    results, 131072 for bf16; chunks of 4096 are added with a rounding each."""
    g = torch.Generator(device="cuda").manual_seed(N + K)
    off = ref.offsets_of(sizes)
    rows, E = int(off[-1]), len(sizes)
    some = lambda *shape: (1 + torch.rand(*shape, device="cuda", generator=g))  # noqa: E731
    A = (some(rows, K) * 2.0 ** -4).to(dtype)
    B = (some(E, K, N) if transposed else some(E, N, K)).mul_(2.0 ** -8 if K < 1 << 18 else 2.0 ** -12).to(dtype)
    C = torch.zeros(rows, N, device="cuda", dtype=dtype)
    bsfp8.bs16_grouped_gemm(A, B, off.cuda(), C, rows, N, K, E, E, transposed=transposed)
    _no_error()
    for e, (r0, r1) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        W = B[e] if transposed else B[e].t()
        want = sum(A[r0:r1, k: k + 8192].double() @ W[k: k + 8192].double() for k in range(0, K, 8192))
        most = 16384 if dtype is FP16 else 131072
        tol = want * ((min(K, most) / 16 + 2) * 2.0 ** -23 + K / 4096 * 2.0 ** -24)
        off_by = (C[r0:r1].double() - want).abs()
        assert torch.all(off_by <= tol + (want + tol) * ref.HALF[dtype]), float((off_by / want).max())


# ------------------------------------------------------------------------------ SwiGLU's gradient in fp32
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_swiglu_backward_before_it_is_rounded(dtype):
    """A block of 128 with one value that is not zero has the scale value / 448 in fp32: the gradient
    before it is rounded.  In units of 2^-24, with u = d = 1: exp 4 (2 units in the last place), 1 + e
    1, the reciprocal 2, so s 7; d_u two more for the product and 1 / 448: 9.  1 - s is e s (4 + 7 + 1)
    or the difference (8 of it), with 1 in between and three roundings around it: 7 + 12 + 4 of d_g's
    terms."""
    g = torch.linspace(-80, 80, 64 * 512).to(dtype).view(512, 64)  # 512 rows of 64 blocks
    rows, N = g.shape[0], 64 * 128
    h = torch.zeros(rows, 2 * N, dtype=dtype)
    d = torch.zeros(rows, N, dtype=dtype)
    h[:, :N: 128], h[:, N:: 128], d[:, ::128] = g, 1.0, 1.0
    q, scales = torch.zeros(rows, 2 * N, dtype=torch.uint8, device="cuda"), torch.zeros(2 * N // 128, rows, device="cuda")
    bsfp8.bsmx_swiglu_backward(h.cuda(), d.cuda(), rows, N, q=q, scales=scales, format="blockwise")
    _no_error()
    d_g, d_u = (scales.t().double().cpu() * 448).chunk(2, dim=1)
    x = g.double()
    s, r = torch.special.expit(x), torch.special.expit(-x)
    want_g, want_u, unit = (s * (1 + x * r)).abs(), (x * s).abs(), 2.0 ** -24
    want_u = torch.where(x == 0, torch.full_like(x, 448.0), want_u)  # a block of zeros has scale 1
    assert torch.all((d_u - want_u).abs() <= 9 * unit * want_u), float(((d_u - want_u).abs() / want_u).max() / unit)
    off_by = (d_g - want_g).abs() / (s * (1 + x.abs() * r))
    assert torch.all(off_by <= 23 * unit), float(off_by.max() / unit)


# ------------------------------------------------------------------------------ every form, turning
@pytest.mark.parametrize("transposed", [False, True])
def test_every_product_form_is_taken_on_this_device(transposed):
    """(Which sizes take which is pinned for the usual numbers of clusters: test_expert_plan.py.)"""
    taken = set()
    for _, _, sizes, N, K in forms.PRODUCTS:
        p = bsfp8.bs16_grouped_gemm_plan(sum(sizes), N, K, len(sizes), transposed=transposed, clusters=None)
        taken.add((p["tile_rows"], p["k_shared_by"]))
    assert taken == {(rows, shared) for rows, shared, *_ in forms.PRODUCTS}


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("case", forms.PRODUCTS, ids=lambda c: f"{c[0]}by{c[1]}-{sum(c[2])}in{len(c[2])}-{c[3]}-{c[4]}")
def test_product_forms(case, transposed):
    _, _, sizes, N, K = case
    (off, groups), M, E, spare = _groups(sizes), sum(sizes), len(sizes), 5
    dtype = BF16 if N % 16 else FP16
    A, B = _rand(1, M, K, dtype=dtype), _rand(2, *((E, K, N) if transposed else (E, N, K)), dtype=dtype, scale=K ** -0.5)
    C = torch.full((M + spare, N), 7.0, dtype=dtype, device="cuda")
    bsfp8.bs16_grouped_gemm(A, B, off, C, M, N, K, E, E, transposed=transposed)
    _no_error()
    assert torch.all(C[M:] == 7)
    for e, (r0, r1) in groups:
        x, W = A[r0:r1].double(), (B[e] if transposed else B[e].t()).double()
        _close(C[r0:r1], x @ W, (x.abs() @ W.abs()) * (K / 16 + 2) * 2.0 ** -23, dtype)


@pytest.mark.parametrize("transposed", [False, True])
def test_product_in_chunks_over_several_tiles(transposed):
    sizes, N, K = [700, 300, 0, 257, 1, 16], 4104, 16456
    assert bsfp8.bs16_grouped_gemm_plan(sum(sizes), N, K, len(sizes), transposed=transposed, type="fp16", clusters=None)["k_chunk"] == 4096
    (off, groups), M, E = _groups(sizes), sum(sizes), len(sizes)
    A, B = _rand(1, M, K, dtype=FP16), _rand(2, *((E, K, N) if transposed else (E, N, K)), dtype=FP16, scale=K ** -0.5)
    C = torch.zeros(M, N, dtype=FP16, device="cuda")
    bsfp8.bs16_grouped_gemm(A, B, off, C, M, N, K, E, E, transposed=transposed)
    _no_error()
    for e, (r0, r1) in groups:
        x, W = A[r0:r1].double(), (B[e] if transposed else B[e].t()).double()
        _close(C[r0:r1], x @ W, (x.abs() @ W.abs()) * (4096 / 16 + 2 + 5) * 2.0 ** -23, FP16)


def _check_gradients(dB, values, groups, plus, out, step):
    for e, (r0, r1) in groups:
        x, y = values(r0, r1, e)
        T = x.abs().t() @ y.abs()
        want, tol = x.t() @ y, T * ((r1 - r0) / step + 6) * 2.0 ** -23
        if plus is not None:
            want, tol = want + plus[e].double(), tol + (plus[e].double().abs() + T) * 2.0 ** -24
        _close(dB[e], want, tol, out)


@pytest.mark.parametrize("case", forms.GRADIENTS_16, ids=lambda c: f"{c[0]}-{c[1]}-{'added-' if c[2] else ''}{c[3]}-{'tma' if c[4] else 'straight'}-{c[6]}-{c[7]}")
def test_wgrad_forms(case):
    type_, out, added, rows, tma, sizes, N, K = case
    p = bsfp8.bsfp8_grouped_wgrad_plan(sum(sizes), N, K, len(sizes), fp8=False, out_type=out, added=added, clusters_of_8=None)
    assert p == dict(stage_rows=rows, rows_shared_by=1, stored_by_tma=tma)
    (off, groups), M, E, spare, dtype, out = _groups(sizes), sum(sizes), len(sizes), 3, TYPES[type_], TYPES[out]
    dC, A = _rand(1, M + spare, N, dtype=dtype), _rand(2, M + spare, K, dtype=dtype)
    dC[M:], A[M:] = float("nan"), float("inf")
    plus = _rand(3, E, N, K, dtype=out, scale=3.0) if added else None
    whole = torch.full((E * N * K + 256,), 7.0, dtype=out, device="cuda")
    dB = whole[: E * N * K].view(E, N, K)
    if added:
        dB.copy_(plus)
    bsfp8.bs16_grouped_wgrad(dC, A, off, dB, M + spare, N, K, E, add=dB if added else None)
    _no_error()
    assert torch.all(whole[E * N * K:] == 7)
    _check_gradients(dB, lambda r0, r1, e: (dC[r0:r1].double(), A[r0:r1].double()), groups, plus, out, 16)


@pytest.mark.parametrize("case", forms.GRADIENTS_8, ids=lambda c: f"{c[0]}-{'added-' if c[1] else ''}{'tma' if c[2] else 'straight'}-{sum(c[3])}-{c[4]}-{c[5]}")
def test_wgrad8_forms(case):
    out, added, tma, sizes, N, K = case
    p = bsfp8.bsfp8_grouped_wgrad_plan(sum(sizes), N, K, len(sizes), fp8=True, out_type=out, added=added, clusters_of_8=None)
    assert p == dict(stage_rows=128, rows_shared_by=1, stored_by_tma=tma)
    (off, groups), M, E, spare, out = _groups(sizes), sum(sizes), len(sizes), 3, TYPES[out]
    used = torch.zeros((M + spare) // 128 + E, dtype=torch.bool, device="cuda")
    used[[s for s, _, _ in ref.blocks_of(off.cpu())]] = True

    def operand(seed, n):
        q = _rand(seed, M + spare, n, dtype=FP32, scale=20.0).to(ref.E4M3).view(torch.uint8)
        q[M:] = 0x7F  # NaN
        s = torch.exp(_rand(seed + 9, used.numel(), n, dtype=FP32)) * 0.01
        s[~used] = float("nan")
        return q, s

    (dC, sc), (A, sa) = operand(1, N), operand(2, K)
    plus = _rand(3, E, N, K, dtype=out, scale=3.0) if added else None
    whole = torch.full((E * N * K + 256,), 7.0, dtype=out, device="cuda")
    dB = whole[: E * N * K].view(E, N, K)
    if added:
        dB.copy_(plus)
    bsfp8.bsfp8_grouped_wgrad(dC, A, sc, sa, off, dB, M + spare, N, K, E, add=dB if added else None)
    _no_error()
    assert torch.all(whole[E * N * K:] == 7)

    def values(r0, r1, e):
        first, blocks = r0 // 128 + e, -(-(r1 - r0) // 128)
        wide = lambda s: s[first: first + blocks].double().repeat_interleave(128, 0)[: r1 - r0]  # noqa: E731
        return dC[r0:r1].view(ref.E4M3).double() * wide(sc), A[r0:r1].view(ref.E4M3).double() * wide(sa)

    _check_gradients(dB, values, groups, plus, out, 32)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("top_k", [0, 1, 8])
@pytest.mark.parametrize("sizes,K", [([1500, 0, 129, 1371], 7168), ([5000, 1, 0, 3990, 128, 256], 4096), ([2432, 0, 3000], 384)], ids=str)
def test_columns_over_many_tiles(sizes, K, top_k, dtype):
    """A block of threads walks over several tiles of columns.  The definition in fp32, bit for bit: one
    division for the scale, one for its reciprocal, one product, one rounding."""
    off, groups = _groups(sizes)
    kept, E = sum(sizes), len(sizes)
    M = -(-(kept + 40) // 8) * 8
    x = _rand(K + kept, M // max(top_k, 1), K, dtype=FP32)
    x = (x * torch.exp(_rand(4, 1, K, dtype=FP32))).to(dtype)
    slot = None
    rows = x
    if top_k:
        slot = torch.randperm(M, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.int32)
        slot[torch.arange(0, kept, 97, device="cuda")] = -1
        slot[kept:] = -1
        rows = x[slot.clamp(min=0).long() // top_k]
        rows[slot < 0] = 0
    else:
        x[kept:] = float("nan")
    q = torch.full((M, K), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((M // 128 + E, K), 7.0, device="cuda")
    bsfp8.bsfp8_quantize_columns(x, off, q, s, M, K, E, slot_of_row=slot, top_k=max(top_k, 1))
    _no_error()
    want_s, want_q = torch.full_like(s, 7.0), torch.full_like(q, 7)
    for b, r0, r1 in ref.blocks_of(off.cpu()):
        v = rows[r0:r1].float()
        a = v.abs().amax(0)
        want_s[b] = torch.where(a == 0, torch.ones_like(a), (a / torch.full_like(a, 448.0)).clamp(min=2.0 ** -126))
        want_q[r0:r1] = (v * (torch.ones_like(a) / want_s[b])).clamp(-448, 448).to(ref.E4M3).view(torch.uint8)
    assert torch.equal(s, want_s)
    assert torch.equal(q, want_q)


def test_same_bits_every_time_in_long_loops():
    sizes, N, K = forms.LONG, 512, 1024
    (off, _), M, E = _groups(sizes), sum(sizes), len(sizes)
    x, y = _rand(1, M, N), _rand(2, M, K)
    W = _rand(3, E, N, K, scale=0.05)
    qx, sx = torch.zeros(M, N, dtype=torch.uint8, device="cuda"), torch.zeros(M // 128 + E, N, device="cuda")
    qy, sy = torch.zeros(M, K, dtype=torch.uint8, device="cuda"), torch.zeros(M // 128 + E, K, device="cuda")
    runs = []
    for _ in range(4):
        C = torch.full((M, N), 3.0, dtype=BF16, device="cuda")
        dB, dB8 = (torch.full((E, N, K), 3.0, device="cuda") for _ in range(2))
        bsfp8.bs16_grouped_gemm(y, W, off, C, M, N, K, E, E)
        bsfp8.bs16_grouped_wgrad(x, y, off, dB, M, N, K, E)
        bsfp8.bsfp8_quantize_columns(C, off, qx, sx, M, N, E)
        bsfp8.bsfp8_quantize_columns(y, off, qy, sy, M, K, E)
        bsfp8.bsfp8_grouped_wgrad(qx, qy, sx, sy, off, dB8, M, N, K, E)
        runs.append([t.clone() for t in (C, dB, dB8, qx, sx, qy, sy)])
    _no_error()
    for later in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], later))


# ------------------------------------------------------------------------------ a step of no tokens
@pytest.mark.parametrize("fmt", ["bf16", "blockwise"])
def test_step_without_tokens(fmt):
    import moe_training
    y, ids, weights, gate_up, down, d_out = moe_training.random_step(4, 256, 128, 3, 2)
    experts = moe_training.TrainedExperts(gate_up, down, 2, fmt, max_rows=4)
    experts.d_gate_up.fill_(1.5)
    out, kept = experts.forward(y[:0], ids[:0], weights[:0])
    d_y, d_weights = experts.backward(d_out[:0], kept)
    _no_error()
    assert out.shape == d_y.shape == (0, 256) and d_weights.shape == (0, 2)
    assert torch.all(experts.d_gate_up == 1.5) and torch.all(experts.d_down == 0)
