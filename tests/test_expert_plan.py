"""The rules that choose the experts' kernels, on the host: the sizes of expert_forms.py take the forms
that they stand for, the limits of one accumulator, and what the queries refuse."""
import ctypes

import pytest

import block_scaled_fp8_persistent_gb300 as bsfp8
import expert_forms as forms
from block_scaled_fp8_persistent_gb300 import build as libbuild

NULL, SHAPE, FORMAT = 1, 2, 9


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()


@pytest.mark.parametrize("transposed", [False, True])
def test_products_take_the_forms_they_stand_for(transposed):
    for rows, shared, sizes, N, K in forms.PRODUCTS:
        p = bsfp8.bs16_grouped_gemm_plan(sum(sizes), N, K, len(sizes), transposed=transposed)
        few = rows == 32
        assert p == dict(tile_rows=rows, tile_cols=128 if few else 256, ctas_per_tile=1 if few else 2, k_shared_by=shared, k_chunk=0), (sizes, N, K)
    taken = {(rows, shared) for rows, shared, *_ in forms.PRODUCTS}
    assert taken == {(32, 1), (32, 2), (32, 4), (32, 8), (64, 1), (128, 1), (128, 2), (128, 4), (256, 1), (512, 1)}


def test_gradients_take_the_forms_they_stand_for():
    for type_, out, added, rows, tma, sizes, N, K in forms.GRADIENTS_16:
        p = bsfp8.bsfp8_grouped_wgrad_plan(sum(sizes), N, K, len(sizes), fp8=False, out_type=out, added=added)
        assert p == dict(stage_rows=rows, rows_shared_by=1, stored_by_tma=tma), (out, added, N, K)
    for out, added, tma, sizes, N, K in forms.GRADIENTS_8:
        p = bsfp8.bsfp8_grouped_wgrad_plan(sum(sizes), N, K, len(sizes), fp8=True, out_type=out, added=added)
        assert p == dict(stage_rows=128, rows_shared_by=1, stored_by_tma=tma), (out, added, N, K)
    for sizes, N, K in (([9000], 264, 136), ([2900, 3, 0, 1300], 264, 136)):
        for fp8 in (False, True):
            p = bsfp8.bsfp8_grouped_wgrad_plan(sum(sizes), N // 128 * 128, K // 128 * 128, len(sizes), fp8=fp8)
            assert p == dict(stage_rows=128, rows_shared_by=4, stored_by_tma=False)


@pytest.mark.parametrize("type,most", [("fp16", 16384), ("bf16", 131072)])
@pytest.mark.parametrize("rows", [1, 20, 300, 5000])
@pytest.mark.parametrize("N", [64, 512, 4096, 8192])
def test_no_accumulator_takes_more_of_k_than_it_may(type, most, rows, N):
    for K in (most, most + 8, 2 * most, 8 * most, 8 * most + 64, 1 << 24):
        p = bsfp8.bs16_grouped_gemm_plan(rows, N, K, 1, type=type)
        part = -(-(-(-K // 64)) // p["k_shared_by"]) * 64
        assert (p["k_chunk"] or part) <= most, (K, p)
        assert p["k_chunk"] in (0, 4096) and (K > most or not p["k_chunk"])


def test_refusals():
    lib, out = bsfp8.load_library(), (ctypes.c_int32 * 5)()
    held = (ctypes.c_int32 * 3)(76, 36, 15)
    product = lambda t=0, M=10, N=64, K=64, G=1, sms=152, to=out: lib.bs16_grouped_gemm_plan(t, 0, M, N, K, G, sms, held, to)  # noqa: E731
    assert product() == 0 and product(to=None) == NULL and product(t=2) == FORMAT
    for bad in (dict(M=0), dict(M=1 << 31), dict(N=4), dict(K=12), dict(G=0), dict(sms=1)):
        assert product(**bad) == SHAPE, bad
    grad = lambda f=0, o=2, M=10, N=64, K=64, E=1, sms=152, to=out: lib.bsfp8_grouped_wgrad_plan(f, o, 0, M, N, K, E, sms, 15, to)  # noqa: E731
    assert grad() == 0 and grad(M=0) == 0 and grad(to=None) == NULL and grad(o=3) == FORMAT
    for bad in (dict(M=-1), dict(N=4), dict(f=1), dict(E=0), dict(sms=0)):
        assert grad(**bad) == SHAPE, bad
    with pytest.raises(bsfp8.BsFp8Error):
        bsfp8.bs16_grouped_gemm_plan(10, 12, 64, 1)
    with pytest.raises(bsfp8.BsFp8Error):
        bsfp8.bsfp8_grouped_wgrad_plan(10, 64, 64, 1, fp8=True)


def test_gathering_no_rows_is_no_error():
    """An empty map's address is NULL: with no rows that is not a map that is missing.  (Past the checks
    the call wants a device.)"""
    lib, FAKE = bsfp8.load_library(), 1 << 20
    columns = lambda M, k: lib.bsfp8_quantize_columns(0, FAKE, None, k, FAKE, FAKE, FAKE, M, 4, 256, 2, None)  # noqa: E731
    quantize = lambda rows, k: lib.bsmx_quantize(3, 0, FAKE, None, k, FAKE, FAKE, rows, 4, 256, None)  # noqa: E731
    for call in (columns, quantize):
        assert call(0, 8) != SHAPE and call(0, 1) != SHAPE
        assert call(2, 8) == SHAPE and call(2, 1) == SHAPE and call(0, 0) == SHAPE
