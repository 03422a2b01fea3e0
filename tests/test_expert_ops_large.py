"""The experts' operators on operands of more than 2^31 elements and of more than 2^32 bytes, whose
last rows or experts are compared with 64-bit products (tolerances as in test_expert_ops.py)."""
import pytest
import torch

import block_scaled_fp8_persistent_gb300 as bsfp8
import expert_reference as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=BF16)


def _close(got, want, tol, dtype):
    got, want, tol = got.double(), want.double(), tol.double()
    assert torch.all((got - want).abs() <= tol + (want.abs() + tol) * ref.HALF[dtype])
    assert bsfp8.bsfp8_get_device_error() == 0


def _product(x, W):
    return x.double() @ W.double(), x.double().abs() @ W.double().abs()


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("sizes", [[0] * 518 + [3, 2], [0] * 518 + [130, 70]], ids=["few", "more"])
def test_product_many_weights(sizes, transposed):
    E, N, K = len(sizes), 2048, 2056
    rows = sum(sizes)
    A, B = _rand(1, rows, K), _rand(2, *((E, K, N) if transposed else (E, N, K)))
    assert B.numel() > 2 ** 31
    C = torch.empty(rows, N, device="cuda", dtype=BF16)
    bsfp8.bs16_grouped_gemm(A, B, ref.offsets_of(sizes).cuda(), C, rows, N, K, E, E, transposed=transposed)
    at = 0
    for e in (E - 2, E - 1):
        want, T = _product(A[at: at + sizes[e]], B[e] if transposed else B[e].t())
        _close(C[at: at + sizes[e]], want, T * (K / 16 + 2) * 2.0 ** -23, BF16)
        at += sizes[e]


@pytest.mark.parametrize("transposed", [False, True])
def test_product_many_rows(transposed):
    rows, N, K, E = 1_100_000, 2048, 64, 3
    sizes = [7, rows - 300 - 7, 300]
    A = _rand(1, rows, K)
    B, C = _rand(2, *((E, K, N) if transposed else (E, N, K))), torch.empty(rows, N, device="cuda", dtype=BF16)
    assert C.numel() > 2 ** 31
    bsfp8.bs16_grouped_gemm(A, B, ref.offsets_of(sizes).cuda(), C, rows, N, K, E, E, transposed=transposed)
    for r0, r1, e in ((0, 7, 0), (7, 500, 1), (rows - 900, rows - 300, 1), (rows - 300, rows, 2)):
        want, T = _product(A[r0:r1], B[e] if transposed else B[e].t())
        _close(C[r0:r1], want, T * (K / 16 + 2) * 2.0 ** -23, BF16)


def test_product_rows_far_into_a():
    rows, N, K = 1_100_000, 64, 2048
    sizes = [rows - 40, 40]
    A, B = _rand(1, rows, K), _rand(2, 2, N, K)
    assert A.numel() > 2 ** 31
    C = torch.empty(rows, N, device="cuda", dtype=BF16)
    bsfp8.bs16_grouped_gemm(A, B, ref.offsets_of(sizes).cuda(), C, rows, N, K, 2, 2)
    for r0, r1, e in ((rows - 600, rows - 40, 0), (rows - 40, rows, 1)):
        want, T = _product(A[r0:r1], B[e].t())
        _close(C[r0:r1], want, T * (K / 16 + 2) * 2.0 ** -23, BF16)


@pytest.mark.parametrize("out", [BF16, torch.float32])
def test_wgrad_many_gradients(out):
    E, N, K = 520, 2048, 2056
    sizes = [0] * (E - 2) + [33, 90]
    rows = sum(sizes)
    dC, A = _rand(1, rows, N), _rand(2, rows, K)
    dB = torch.empty(E, N, K, device="cuda", dtype=out)
    assert dB.numel() > 2 ** 31
    bsfp8.bs16_grouped_wgrad(dC, A, ref.offsets_of(sizes).cuda(), dB, rows, N, K, E)
    for e, r0, r1 in ((E - 2, 0, 33), (E - 1, 33, 123)):
        want, T = _product(dC[r0:r1].t(), A[r0:r1])
        _close(dB[e], want, T * (90 / 16 + 2) * 2.0 ** -23, out)
    assert all(int(torch.count_nonzero(dB[e0: min(e0 + 64, E - 2)])) == 0 for e0 in range(0, E - 2, 64))


def test_wgrad_rows_far_down():
    rows, N, K = 1_100_000, 2048, 64
    sizes = [rows - 77, 77]
    dC, A = _rand(1, rows, N), _rand(2, rows, K)
    assert dC.numel() > 2 ** 31
    dB = torch.empty(2, N, K, device="cuda")
    bsfp8.bs16_grouped_wgrad(dC, A, ref.offsets_of(sizes).cuda(), dB, rows, N, K, 2)
    want, T = _product(dC[rows - 77:].t(), A[rows - 77:])
    _close(dB[1], want, T * (77 / 16 + 2) * 2.0 ** -23, torch.float32)
    want, T = torch.zeros(N, K, device="cuda", dtype=torch.float64), torch.zeros(N, K, device="cuda", dtype=torch.float64)
    for r in range(0, rows - 77, 100_000):
        w, t = _product(dC[r: min(r + 100_000, rows - 77)].t(), A[r: min(r + 100_000, rows - 77)])
        want += w
        T += t
    _close(dB[0], want, T * (rows / 16) * 2.0 ** -23, torch.float32)
    # nearer than that bound: chunks of 512 rows are exact to 32 additions, and 2149 of them follow
    assert float((dB[0].double() - want).norm() / want.norm()) < 2149 * 2.0 ** -24 + 34 * 2.0 ** -23


def test_columns_and_fp8_wgrad_rows_far_down():
    rows, N, K = 2_200_000, 1024, 128
    sizes = [rows - 200, 200]
    off = ref.offsets_of(sizes).cuda()
    x, z = _rand(1, rows, N), _rand(2, rows, K)
    assert x.numel() > 2 ** 31
    quantised = []
    for t, n in ((x, N), (z, K)):
        q = torch.empty(rows, n, dtype=torch.uint8, device="cuda")
        s = torch.empty(rows // 128 + 2, n, device="cuda")
        bsfp8.bsfp8_quantize_columns(t, off, q, s, rows, n, 2)
        quantised.append((q, s))
    first = sizes[0] // 128 + 1  # the second group's first row of scales
    values = []
    for (q, s), t in zip(quantised, (x, z)):
        tail = t[rows - 200:].double()
        scale = torch.cat([s[first].expand(128, -1), s[first + 1].expand(72, -1)]).double()
        v = q[rows - 200:].view(torch.float8_e4m3fn).double() * scale
        assert torch.all((v - tail).abs() <= (tail.abs() * 2.0 ** -4).maximum(scale * 2.0 ** -10) * (1 + 2.0 ** -17))
        values.append(v)
    dB = torch.empty(2, N, K, device="cuda")
    bsfp8.bsfp8_grouped_wgrad(quantised[0][0], quantised[1][0], quantised[0][1], quantised[1][1], off, dB, rows, N, K, 2)
    want, T = _product(values[0].t(), values[1])
    _close(dB[1], want, T * (200 / 32 + 6) * 2.0 ** -23, torch.float32)


def test_swiglu_gradient_rows_far_down():
    rows, N = 540_000, 2048
    h, d = _rand(1, rows, 2 * N), _rand(2, rows, N)
    assert h.numel() > 2 ** 31
    act = torch.empty(rows, N, device="cuda", dtype=BF16)
    q, s = torch.empty(rows, 2 * N, dtype=torch.uint8, device="cuda"), torch.empty(2 * N // 128, rows, device="cuda")
    bsfp8.bsmx_swiglu_backward(h, d, rows, N, d_h=h, act=act, q=q, scales=s)  # d_h in place
    h2 = _rand(1, rows, 2 * N)[-3:].cpu()
    want_act, want, mag = ref.swiglu_backward(h2, d[-3:].cpu())
    g = h2[:, :N].double().abs()
    u = (10 + g) * 2.0 ** -22
    _close(act[-3:].cpu(), want_act, want_act.abs() * u, BF16)
    terms = mag * torch.cat([u * (1 + g), u], dim=1)
    _close(h[-3:].cpu(), want, terms, BF16)
    scale = s[:, -3:].t().double().cpu().repeat_interleave(128, 1)
    v = q[-3:].cpu().view(torch.float8_e4m3fn).double() * scale
    assert torch.all((v - want).abs() <= (want.abs() * 2.0 ** -4).maximum(scale * 2.0 ** -10) * (1 + 2.0 ** -17) + terms * 1.1)
