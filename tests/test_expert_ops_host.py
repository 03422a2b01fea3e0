"""The experts' products in 16 bits and the backward pass of the experts on the host: what is
refused before any GPU work, and the 64-bit definitions the GPU tests compare with."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_persistent_gb300 as bsfp8
import expert_reference as ref
from block_scaled_fp8_persistent_gb300 import build as libbuild

FAKE = 1 << 20  # a 32-byte aligned non-null address; never dereferenced on these paths
NULL, SHAPE, ALIGN, FORMAT = 1, 2, 3, 9


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return bsfp8.load_library()


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), FORMAT), (dict(t=-1), FORMAT),
    (dict(off=None), NULL), (dict(B=None), NULL), (dict(A=None), NULL), (dict(C=None), NULL),
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(N=0), SHAPE), (dict(N=12), SHAPE), (dict(N=-8), SHAPE),
    (dict(K=0), SHAPE), (dict(K=4), SHAPE), (dict(K=(1 << 24) + 8), SHAPE), (dict(N=1 << 20, K=1 << 18), SHAPE),
    (dict(G=0), SHAPE), (dict(E=0), SHAPE), (dict(G=3, ids=None), SHAPE), (dict(G=(1 << 20) + 1), SHAPE),
    (dict(A=FAKE + 8), ALIGN), (dict(B=FAKE + 8), ALIGN), (dict(C=FAKE + 8), ALIGN), (dict(off=FAKE + 2), ALIGN),
    (dict(ids=FAKE + 2), ALIGN),
])
@pytest.mark.parametrize("transposed", [0, 1])
def test_product_refusals(lib, kw, status, transposed):
    a = dict(t=0, A=FAKE, B=FAKE, off=FAKE, ids=FAKE, C=FAKE, M=10, N=64, K=128, G=2, E=2)
    a.update(kw)
    assert lib.bs16_grouped_gemm(a["t"], transposed, a["A"], a["B"], a["off"], a["ids"], a["C"], a["M"], a["N"], a["K"],
                                 a["G"], a["E"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), FORMAT), (dict(out=1), FORMAT), (dict(t=1, out=0), FORMAT), (dict(out=3), FORMAT),
    (dict(dC=None), NULL), (dict(A=None), NULL), (dict(off=None), NULL), (dict(dB=None), NULL),
    (dict(M=0, dB=None), NULL),
    (dict(M=-1), SHAPE), (dict(N=4), SHAPE), (dict(K=12), SHAPE), (dict(E=0), SHAPE), (dict(N=1 << 20, K=1 << 18), SHAPE),
    (dict(dC=FAKE + 8), ALIGN), (dict(A=FAKE + 8), ALIGN), (dict(add=FAKE + 8), ALIGN), (dict(dB=FAKE + 8), ALIGN),
    (dict(off=FAKE + 1), ALIGN),
])
def test_wgrad_refusals(lib, kw, status):
    a = dict(t=0, out=2, dC=FAKE, A=FAKE, off=FAKE, add=None, dB=FAKE, M=10, N=64, K=128, E=2)
    a.update(kw)
    assert lib.bs16_grouped_wgrad(a["t"], a["out"], a["dC"], a["A"], a["off"], a["add"], a["dB"], a["M"], a["N"], a["K"],
                                  a["E"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(out=3), FORMAT), (dict(out=-1), FORMAT),
    (dict(dC=None), NULL), (dict(A=None), NULL), (dict(sc=None), NULL), (dict(sa=None), NULL), (dict(off=None), NULL),
    (dict(dB=None), NULL),
    (dict(N=64), SHAPE), (dict(K=192), SHAPE), (dict(M=1 << 31), SHAPE), (dict(E=0), SHAPE),
    (dict(dC=FAKE + 8), ALIGN), (dict(A=FAKE + 8), ALIGN), (dict(sc=FAKE + 2), ALIGN), (dict(sa=FAKE + 4), ALIGN),
    (dict(add=FAKE + 8), ALIGN), (dict(dB=FAKE + 8), ALIGN),
])
def test_wgrad8_refusals(lib, kw, status):
    a = dict(out=2, dC=FAKE, A=FAKE, sc=FAKE, sa=FAKE, off=FAKE, add=None, dB=FAKE, M=10, N=128, K=256, E=2)
    a.update(kw)
    assert lib.bsfp8_grouped_wgrad(a["out"], a["dC"], a["A"], a["sc"], a["sa"], a["off"], a["add"], a["dB"], a["M"], a["N"],
                                   a["K"], a["E"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(t=3), FORMAT), (dict(t=-1), FORMAT),
    (dict(x=None), NULL), (dict(off=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL),
    (dict(K=64), SHAPE), (dict(K=(1 << 22) + 128), SHAPE), (dict(M=-1, xr=-1), SHAPE), (dict(xr=9), SHAPE), (dict(k=2), SHAPE),
    (dict(map=FAKE, k=0), SHAPE), (dict(map=FAKE, k=65), SHAPE), (dict(map=FAKE, xr=-1), SHAPE), (dict(G=0), SHAPE),
    (dict(x=FAKE + 8), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(s=FAKE + 4), ALIGN), (dict(map=FAKE + 2), ALIGN),
])
def test_columns_refusals(lib, kw, status):
    a = dict(t=0, x=FAKE, map=None, k=1, off=FAKE, q=FAKE, s=FAKE, M=10, xr=10, K=256, G=2)
    a.update(kw)
    assert lib.bsfp8_quantize_columns(a["t"], a["x"], a["map"], a["k"], a["off"], a["q"], a["s"], a["M"], a["xr"], a["K"],
                                      a["G"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), FORMAT), (dict(fmt=4), FORMAT), (dict(fmt=-1), FORMAT),
    (dict(h=None), NULL), (dict(d=None), NULL), (dict(dh=None, act=None, q=None), NULL), (dict(s=None), NULL),
    (dict(dh=None, d=None), NULL), (dict(q=None, d=None), NULL),
    (dict(N=64), SHAPE), (dict(N=200), SHAPE), (dict(N=(1 << 23) + 128), SHAPE), (dict(rows=-1), SHAPE),
    (dict(rows=(1 << 31) - 1, N=1 << 22), SHAPE),
    (dict(h=FAKE + 8), ALIGN), (dict(d=FAKE + 8), ALIGN), (dict(dh=FAKE + 8), ALIGN), (dict(act=FAKE + 8), ALIGN),
    (dict(q=FAKE + 8), ALIGN), (dict(fmt=3, s=FAKE + 2), ALIGN),
])
def test_swiglu_backward_refusals(lib, kw, status):
    a = dict(t=0, fmt=0, h=FAKE, d=FAKE, dh=FAKE, act=FAKE, q=FAKE, s=FAKE, rows=5, N=256)
    a.update(kw)
    assert lib.bsmx_swiglu_backward(a["t"], a["fmt"], a["h"], a["d"], a["dh"], a["act"], a["q"], a["s"], a["rows"], a["N"],
                                    None) == status


def test_binding_refuses_host_raw_and_mixed_arguments():
    libbuild.build()
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bsfp8.bs16_grouped_gemm(x, FAKE, FAKE, FAKE, 2, 128, 128, 1, 1)
    with pytest.raises(ValueError, match="type"):
        bsfp8.bs16_grouped_gemm(FAKE, FAKE, FAKE, FAKE, 2, 128, 128, 1, 1)
    with pytest.raises(ValueError, match="unsupported type"):
        bsfp8.bs16_grouped_gemm(x.float(), FAKE, FAKE, FAKE, 2, 128, 128, 1, 1)
    with pytest.raises(ValueError, match="type"):
        bsfp8.bs16_grouped_wgrad(x, FAKE, FAKE, FAKE, 2, 128, 128, 1)  # dB's type is not known
    with pytest.raises(ValueError, match="unsupported type"):
        bsfp8.bsfp8_quantize_columns(x.double(), FAKE, FAKE, FAKE, 2, 128, 1)
    with pytest.raises(ValueError, match="unsupported type"):
        bsfp8.bsmx_swiglu_backward(torch.zeros(2, 256), FAKE, 2, 128, d_h=FAKE)
    with pytest.raises(KeyError):
        bsfp8.bsmx_swiglu_backward(FAKE, FAKE, 2, 128, d_h=FAKE, type="bf16", format="int8")
    with pytest.raises(bsfp8.BsFp8Error) as e:
        bsfp8.bs16_grouped_gemm(FAKE, FAKE, FAKE, FAKE, 2, 100, 128, 1, 1, type="bf16", stream=0)
    assert e.value.status == SHAPE


def test_gathered_rows_are_a_token_for_every_top_k_slots_unless_told_otherwise(monkeypatch):
    import types
    seen = []
    fake = types.SimpleNamespace(quantize_columns=lambda *args: seen.append(args[8]) or 0)  # x_rows
    monkeypatch.setattr(bsfp8, "_binding", fake)
    bsfp8.bsfp8_quantize_columns(FAKE, FAKE, FAKE, FAKE, 40, 128, 1, x_type="bf16")
    bsfp8.bsfp8_quantize_columns(FAKE, FAKE, FAKE, FAKE, 40, 128, 1, x_type="bf16", slot_of_row=FAKE, top_k=8)
    bsfp8.bsfp8_quantize_columns(FAKE, FAKE, FAKE, FAKE, 40, 128, 1, x_type="bf16", slot_of_row=FAKE, top_k=8, x_rows=17)
    assert seen == [40, 5, 17]


# ------------------------------------------------------------------- the 64-bit definitions
def test_blocks_of_any_partition_fit_and_do_not_meet():
    g = np.random.default_rng(1)
    for _ in range(200):
        sizes = g.integers(0, 400, size=g.integers(1, 9)) * g.integers(0, 2, size=1)
        off = ref.offsets_of(sizes.tolist())
        rows = [s for s, _, _ in ref.blocks_of(off)]
        assert len(set(rows)) == len(rows) and all(s < int(off[-1]) // 128 + len(sizes) for s in rows)
        assert sum(r1 - r0 for _, r0, r1 in ref.blocks_of(off)) == int(off[-1])


def test_gradients_are_the_derivative():
    sizes, N, K = [3, 0, 4], 8, 16
    off = ref.offsets_of(sizes)
    A, B, d = (torch.randn(*s, dtype=torch.float64) for s in ((7, K), (3, N, K), (7, N)))
    A.requires_grad_(), B.requires_grad_()
    y = torch.cat([A[r0:r1] @ B[e].t() for e, (r0, r1) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
    (y * d).sum().backward()
    with torch.no_grad():
        assert torch.allclose(ref.product(A, B, off, None, False)[0], y)
        assert torch.allclose(ref.product(d, B, off, None, True)[0], A.grad)
        assert torch.allclose(ref.wgrad(d, A, off)[0], B.grad)


def test_swiglu_gradient_is_the_derivative():
    h, d = torch.randn(3, 32, dtype=torch.float64) * 3, torch.randn(3, 16, dtype=torch.float64)
    act, d_h, _ = ref.swiglu_backward(h, d)
    x = h.clone().requires_grad_()
    g, u = x.chunk(2, dim=1)
    y = g / (1 + torch.exp(-g)) * u
    (y * d).sum().backward()
    assert torch.allclose(act, y.detach()) and torch.allclose(d_h, x.grad)


def test_columns_by_hand():
    x = torch.zeros(130, 128)
    x[0, 0], x[5, 0], x[129, 1] = 448.0, -1.0, 896.0
    q, s = ref.quantise_columns(x, ref.offsets_of([130]))
    v = q.view(ref.E4M3).float()
    assert s[0, 0] == 1 and s[0, 1] == 1 and s[1, 1] == 2 and v[0, 0] == 448 and v[5, 0] == -1 and v[129, 1] == 448


@pytest.mark.parametrize("M,status", [((1 << 31) - 1, SHAPE), ((1 << 31) - 1024, SHAPE), ((1 << 31) - 1025, ALIGN)])
def test_rows_end_before_the_last_tile_would_pass_an_int(lib, M, status):
    # (what is accepted goes on to the alignment)
    bad = FAKE + 8
    assert lib.bs16_grouped_gemm(0, 0, bad, FAKE, FAKE, None, FAKE, M, 8, 8, 1, 1, None) == status
    assert lib.bs16_grouped_wgrad(0, 2, bad, FAKE, FAKE, None, FAKE, M, 8, 8, 1, None) == status
    assert lib.bsfp8_grouped_wgrad(2, bad, FAKE, FAKE, FAKE, FAKE, None, FAKE, M, 128, 128, 1, None) == status
    assert lib.bsfp8_quantize_columns(0, bad, None, 1, FAKE, FAKE, FAKE, M, M, 128, 1, None) == status
