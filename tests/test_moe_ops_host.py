"""The operators around the grouped GEMM on the host: arguments that are refused before any GPU
work, the sort's workspace, and the 64-bit definitions the GPU tests compare with."""
import ctypes
import importlib.machinery
import importlib.util
import os
import re
import shutil
import subprocess
import threading
import time
import types

import numpy as np
import pytest
import torch

import block_scaled_fp8_persistent_gb300 as bsfp8
from block_scaled_fp8_persistent_gb300 import build as libbuild
import moe_reference as ref

FAKE = 1 << 20  # a 32-byte aligned non-null address; never dereferenced on these paths
NULL, SHAPE, ALIGN, FORMAT = 1, 2, 3, 9


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return bsfp8.load_library()


def _quantize(lib, **kw):
    a = dict(fmt=0, xt=0, x=FAKE, map=None, k=1, q=FAKE, s=FAKE, rows=5, out=5, K=256)
    a.update(kw)
    return lib.bsmx_quantize(a["fmt"], a["xt"], a["x"], a["map"], a["k"], a["q"], a["s"],
                             a["rows"], a["out"], a["K"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=4), FORMAT), (dict(fmt=-1), FORMAT), (dict(xt=3), FORMAT),
    (dict(x=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL),
    (dict(K=0), SHAPE), (dict(K=64), SHAPE), (dict(K=200), SHAPE), (dict(rows=-1), SHAPE),
    (dict(K=(1 << 24) + 128), SHAPE), (dict(rows=1 << 31, out=1 << 31), SHAPE), (dict(out=6), SHAPE), (dict(k=2), SHAPE),
    (dict(map=FAKE, k=0), SHAPE), (dict(map=FAKE, k=65), SHAPE),
    (dict(map=FAKE, k=64, rows=1 << 26), SHAPE), (dict(map=FAKE, k=2, out=-1), SHAPE),
    (dict(x=FAKE + 8), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(fmt=3, s=FAKE + 2), ALIGN),
    (dict(map=FAKE + 2, k=2, out=10), ALIGN),
])
def test_quantize_refusals(lib, kw, status):
    assert _quantize(lib, **kw) == status


def _norm(lib, **kw):
    a = dict(fmt=0, rt=0, x=FAKE, r=FAKE, w=FAKE, eps=1e-6, ro=FAKE, y=FAKE, q=FAKE, s=FAKE,
             rows=3, K=256)
    a.update(kw)
    return lib.bsmx_rmsnorm_quant(a["fmt"], a["rt"], a["x"], a["r"], a["w"], a["eps"], a["ro"],
                                  a["y"], a["q"], a["s"], a["rows"], a["K"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=4), FORMAT), (dict(rt=1), FORMAT), (dict(rt=3), FORMAT),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(s=None), NULL),
    (dict(ro=None, y=None, q=None), NULL),
    (dict(K=192), SHAPE), (dict(K=32768 + 128), SHAPE), (dict(rows=-1), SHAPE),
    (dict(eps=0.0), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(eps=float("inf")), SHAPE),
    (dict(x=FAKE + 8), ALIGN), (dict(r=FAKE + 8), ALIGN), (dict(w=FAKE + 2), ALIGN),
    (dict(ro=FAKE + 8), ALIGN), (dict(y=FAKE + 8), ALIGN), (dict(q=FAKE + 4), ALIGN),
])
def test_norm_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=4), FORMAT), (dict(h=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL),
    (dict(N=64), SHAPE), (dict(N=1 << 30), SHAPE), (dict(rows=-1), SHAPE),
    (dict(h=FAKE + 8), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(fmt=3, s=FAKE + 1), ALIGN),
])
def test_swiglu_refusals(lib, kw, status):
    a = dict(fmt=0, h=FAKE, q=FAKE, s=FAKE, rows=4, N=256)
    a.update(kw)
    assert lib.bsmx_swiglu_quant(a["fmt"], a["h"], a["q"], a["s"], a["rows"], a["N"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), NULL), (dict(off=None), NULL), (dict(row=None), NULL),
    (dict(rows=50000, ws=None), NULL), (dict(rows=50000, wsb=16), SHAPE),
    (dict(rows=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE), (dict(E=0), SHAPE),
    (dict(E=4097), SHAPE), (dict(rows=1 << 30, k=2), SHAPE),
    (dict(ids=FAKE + 2), ALIGN), (dict(off=FAKE + 2), ALIGN), (dict(row=FAKE + 1), ALIGN),
    (dict(slot=FAKE + 2), ALIGN), (dict(ws=FAKE + 2), ALIGN),
])
def test_sort_refusals(lib, kw, status):
    a = dict(ids=FAKE, off=FAKE, row=FAKE, slot=FAKE, ws=FAKE, wsb=1 << 20, rows=9, k=2, E=8)
    a.update(kw)
    assert lib.bsmx_moe_sort(a["ids"], a["off"], a["row"], a["slot"], a["ws"], a["wsb"], a["rows"],
                             a["k"], a["E"], None) == status


def test_sort_workspace():
    libbuild.build()
    assert bsfp8.bsmx_moe_sort_workspace(1, 1, 8) == 0
    last = 0
    for rows in (1 << 10, 1 << 14, 1 << 18, 1 << 22, 1 << 27):
        need = bsfp8.bsmx_moe_sort_workspace(rows, 8, 256)
        assert last <= need <= 128 * 257 * 4
        last = need
    for bad in ((-1, 1, 8), (1, 0, 8), (1, 1, 0), (1, 1, 4097), (1 << 31, 1, 8)):
        with pytest.raises(bsfp8.BsFp8Error) as e:
            bsfp8.bsmx_moe_sort_workspace(*bad)
        assert e.value.status == SHAPE


@pytest.mark.parametrize("kw,status", [
    (dict(C=None), NULL), (dict(row=None), NULL), (dict(out=None), NULL),
    (dict(N=4), SHAPE), (dict(N=20), SHAPE), (dict(N=(1 << 24) + 8), SHAPE), (dict(k=0), SHAPE),
    (dict(k=65), SHAPE), (dict(rows=-1), SHAPE), (dict(inr=-1), SHAPE), (dict(inr=1 << 31), SHAPE),
    (dict(C=FAKE + 8), ALIGN), (dict(res=FAKE + 8), ALIGN), (dict(out=FAKE + 2), ALIGN),
    (dict(row=FAKE + 2), ALIGN), (dict(w=FAKE + 2), ALIGN),
])
def test_combine_refusals(lib, kw, status):
    a = dict(C=FAKE, row=FAKE, w=FAKE, res=FAKE, out=FAKE, rows=4, inr=8, k=2, N=256)
    a.update(kw)
    assert lib.bsmx_moe_combine(a["C"], a["row"], a["w"], a["res"], a["out"], a["rows"], a["inr"],
                                a["k"], a["N"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(d=None), NULL), (dict(C=None), NULL), (dict(row=None), NULL), (dict(w=None), NULL),
    (dict(dC=None), NULL), (dict(dw=None), NULL), (dict(N=12), SHAPE), (dict(k=65), SHAPE),
    (dict(d=FAKE + 8), ALIGN), (dict(C=FAKE + 8), ALIGN), (dict(dC=FAKE + 8), ALIGN),
    (dict(dw=FAKE + 2), ALIGN),
])
def test_combine_backward_refusals(lib, kw, status):
    a = dict(d=FAKE, C=FAKE, row=FAKE, w=FAKE, dC=FAKE, dw=FAKE, rows=4, inr=8, k=2, N=256)
    a.update(kw)
    assert lib.bsmx_moe_combine_backward(a["d"], a["C"], a["row"], a["w"], a["dC"], a["dw"],
                                         a["rows"], a["inr"], a["k"], a["N"], None) == status


def test_binding_refuses_host_and_raw_arguments():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bsfp8.bsmx_quantize("mxfp8", x, FAKE, FAKE, 2, 128)
    with pytest.raises(ValueError, match="type"):
        bsfp8.bsmx_quantize("mxfp8", FAKE, FAKE, FAKE, 2, 128)
    with pytest.raises(ValueError, match="type"):
        bsfp8.bsmx_quantize("mxfp8", torch.zeros(2, 128, dtype=torch.float64), FAKE, FAKE, 2, 128)
    with pytest.raises(ValueError, match="bf16"):
        bsfp8.bsmx_swiglu_quant("mxfp8", torch.zeros(2, 256), FAKE, FAKE, 2, 128)
    with pytest.raises(ValueError, match="workspace"):
        bsfp8.bsmx_moe_sort(FAKE, FAKE, FAKE, FAKE, 2, 2, 8)
    with pytest.raises(KeyError):
        bsfp8.bsmx_quantize("int8", FAKE, FAKE, FAKE, 2, 128, x_type="bf16")
    libbuild.build()
    with pytest.raises(bsfp8.BsFp8Error) as e:
        bsfp8.bsmx_quantize("mxfp8", FAKE, FAKE, FAKE, 2, 100, x_type="bf16", stream=0)
    assert e.value.status == SHAPE


def test_kernels_wait_before_they_touch_what_others_wrote():
    # a kernel that starts before the one before it has ended may touch its arguments' memory
    # only after its own wait
    csrc = os.path.join(os.path.dirname(bsfp8.__file__), "csrc")
    kernels = 0
    for name in ("moe_route.cu", "moe_quant.cu"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, name)).read())
        for head in re.finditer(r"__global__ void[^;{]*?(\w+_kernel)\((\w+Args) a\b[^{]*\{", text):
            body = text[head.end():]
            body = body[:body.index("\n}\n")]
            waits = [m.start() for m in re.finditer(r"begin_early\(|wait_for_previous\(|quantise_piece<", body)]
            fields = r"\ba\.(ids|offsets|row_of_slot|slot_of_row|workspace|C|weights?|residual\w*|out|d_\w+|dC|x|h|y|q|scales)\b"
            first = re.search(fields + r"|\bplace_segment\(|\bchecked_row\(", body)
            assert waits and waits[0] < first.start(), head.group(1)
            kernels += 1
    assert kernels == 8


def test_operators_that_store_by_row_say_that_rows_are_distinct():
    # the mapped quantisation and the combine's gradient write each named row whole
    header = open(os.path.join(libbuild.INCLUDE, "bsfp8.h")).read()
    flat = re.sub(r"\s*\n \* *", " ", header)
    for name in ("bsmx_quantize", "bsmx_moe_combine_backward"):
        comment = flat[: flat.index(f"bsfp8_status {name}(")].rsplit("/*", 1)[1]
        assert re.search("[Nn]o row is to be named twice", comment), name


def test_sorted_slots_have_distinct_rows():
    ids = np.random.default_rng(2).integers(-1, 9, size=(40, 5))
    row = ref.sort_slots(ids, 8)[1]
    assert len(np.unique(row[row >= 0])) == (row >= 0).sum()


def test_a_row_map_has_a_row_for_every_slot_unless_told_otherwise(monkeypatch):
    seen = []
    fake = types.SimpleNamespace(quantize=lambda *args: seen.append(args[8]) or 0)  # out_rows
    monkeypatch.setattr(bsfp8, "_binding", fake)
    bsfp8.bsmx_quantize("mxfp8", FAKE, FAKE, FAKE, 5, 128, x_type="bf16")
    bsfp8.bsmx_quantize("mxfp8", FAKE, FAKE, FAKE, 5, 128, x_type="bf16", row_of_slot=FAKE, top_k=8)
    bsfp8.bsmx_quantize("mxfp8", FAKE, FAKE, FAKE, 5, 128, x_type="bf16", row_of_slot=FAKE, top_k=8, out_rows=17)
    assert seen == [5, 40, 17]


def test_binding_refuses_tensors_of_another_gpu():
    # tensors without memory, said to be on a GPU that is not the current one
    libbuild.build()
    class Elsewhere(torch.Tensor):
        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise AssertionError("no operation is asked for")

    x, h, ids = (torch.Tensor._make_wrapper_subclass(Elsewhere, (2, n), dtype=t, device="cuda:7")
                 for n, t in ((128, torch.bfloat16), (256, torch.bfloat16), (2, torch.int32)))
    for call in (lambda: bsfp8.bsmx_quantize("mxfp8", x, FAKE, FAKE, 2, 128),
                 lambda: bsfp8.bsmx_swiglu_quant("mxfp8", h, FAKE, FAKE, 2, 128),
                 lambda: bsfp8.bsmx_rmsnorm_quant("mxfp8", x, FAKE, 1e-6, 2, 128, y=FAKE),
                 lambda: bsfp8.bsmx_moe_sort(ids, FAKE, FAKE, None, 2, 2, 8),
                 lambda: bsfp8.bsmx_moe_combine(FAKE, ids, FAKE, 2, 4, 2, 128)):
        with pytest.raises(ValueError, match="GPU 7"):
            call()


STUB = r"""
#include <unistd.h>
extern "C" {
volatile int entered = 0, go_on = 0;
int wait_for_python(int, const void*, void*, void*, long, int, void*) {
  entered = 1;
  for (int i = 0; i < 2000 && !go_on; ++i) usleep(1000);
  return go_on ? 0 : 5;
}
}
"""


def test_calls_run_without_the_interpreter_lock(tmp_path):
    # an entry point that returns once another Python thread has run, or gives up after 2 s
    libbuild.build()
    (tmp_path / "stub.cpp").write_text(STUB)
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", str(tmp_path / "stub.cpp"), "-o", str(tmp_path / "stub.so")], check=True)
    stub = ctypes.CDLL(str(tmp_path / "stub.so"))
    path = shutil.copy(libbuild.binding_path(), tmp_path / "binding.so")  # an instance of its own
    loader = importlib.machinery.ExtensionFileLoader("bsfp8_binding", str(path))
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("bsfp8_binding", path, loader=loader))
    loader.exec_module(module)
    module.bind(*[ctypes.cast(stub.wait_for_python, ctypes.c_void_p).value] * 6)
    got = []
    call = threading.Thread(target=lambda: got.append(module.swiglu_quant(0, FAKE, FAKE, FAKE, 1, 128, 0)))
    call.start()
    entered, go_on = ctypes.c_int.in_dll(stub, "entered"), ctypes.c_int.in_dll(stub, "go_on")
    while not entered.value:
        time.sleep(0.001)
    go_on.value = 1
    call.join()
    assert got == [0]


# ------------------------------------------------------------------- the 64-bit definitions
def test_nearest_against_torch_float8():
    v = np.concatenate([np.linspace(-460, 460, 4001), np.linspace(-0.02, 0.02, 4001)])
    v = np.concatenate([v, (ref.E4M3[1:] + ref.E4M3[:-1]) / 2])  # every tie
    v = v.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(np.clip(v, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.nearest(v, ref.E4M3), want)


def test_nearest_e2m1_by_hand():
    v = np.array([0.25, 0.2501, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.0, -0.75, -2.51])
    want = [0.0, 0.5, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, -1.0, -3.0]
    assert np.array_equal(ref.nearest(v, ref.E2M1), want)


def test_scales_by_hand():
    a = np.array([0.0, 448.0, 449.0, 1.75, 1.76, 3.5, 224.0])
    assert np.array_equal(ref.scale_of(a, "mxfp8"), [1, 1, 2, 2.0 ** -8, 2.0 ** -7, 2.0 ** -7, 0.5])
    assert np.array_equal(ref.scale_of(np.array([6.0, 6.1, 1.5, 1.6]), "mxfp4"), [1, 2, 0.25, 0.5])
    assert np.array_equal(ref.scale_of(np.array([6.0, 6.3, 1e-9, 1e9]), "nvfp4"),
                          [1.0, 1.0, 2.0 ** -9, 448.0])
    assert np.array_equal(ref.scale_of(np.array([0.0, 896.0, 1e-300]), "blockwise"),
                          [1.0, 2.0, 2.0 ** -126])


def test_sort_reference_by_hand():
    off, row, slot = ref.sort_slots(np.array([2, 0, -1, 2, 7, 0]), 3)
    assert off.tolist() == [0, 2, 2, 4, 6]
    assert row.tolist() == [2, 0, -1, 3, -1, 1]
    assert slot.tolist() == [1, 5, 0, 3, -1, -1]


def test_combine_gradient_is_the_derivative():
    g = np.random.default_rng(3)
    C, d = g.normal(size=(6, 16)), g.normal(size=(3, 16))
    row = np.array([[0, 3], [-1, 5], [2, 1]])
    w = g.normal(size=(3, 2))
    dC, dw, _ = ref.combine_backward(d, C, row, w)
    loss = lambda C_, w_: (ref.combine(C_, row, w_, None)[0] * d).sum()  # noqa: E731
    h = 1e-4
    for t in range(3):
        for j in range(2):
            p, m = w.copy(), w.copy()
            p[t, j] += h
            m[t, j] -= h
            assert abs((loss(C, p) - loss(C, m)) / (2 * h) - dw[t, j]) < 1e-8
    for r in (0, 1, 2, 3, 5):
        p, m = C.copy(), C.copy()
        p[r, 7] += h
        m[r, 7] -= h
        assert abs((loss(p, w) - loss(m, w)) / (2 * h) - dC[r, 7]) < 1e-8
    assert np.isnan(dC[4]).all() and dw[1, 0] == 0
