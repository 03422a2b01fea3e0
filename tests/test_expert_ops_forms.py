"""The experts' operators in the forms that their rules choose for ordinary sizes, and in loops that
are long enough to turn: against 64 bits, with the tolerances of test_expert_ops.py."""
import pytest
import torch

import block_scaled_fp8_persistent_gb300 as bsfp8
import expert_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _no_error():
    assert bsfp8.bsfp8_get_device_error() == 0


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
