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
