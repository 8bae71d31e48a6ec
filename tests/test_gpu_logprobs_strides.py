"""Token log probabilities of FP32 logits whose rows, or whose first row, begin 16 bytes
behind a multiple of 32: what the entry point's alignment (16 bytes) allows."""
import pytest
import torch

from test_gpu_step import _check_logprobs, _run_logprobs, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,V,k", [(1, 1001, 20), (7, 1001, 20), (3, 12, 12), (2, 4, 4), (5, 32003, 64), (16, 128255, 20), (600, 9001, 5)])
@pytest.mark.parametrize("front", [0, 4])
def test_rows_16_bytes_off(rows, V, k, front):
    _say("logprobs %d x %d, k %d, first row %d values in" % (rows, V, k, front))
    ld = (V + 3) // 8 * 8 + 4                                      # 4 mod 8 values, at least V
    assert ld >= V and ld % 8 == 4
    g = torch.Generator(device="cuda").manual_seed(V)
    all_ = torch.full((front + rows * ld,), float("nan"), device="cuda")
    x = all_[front:].view(rows, ld)[:, :V]
    x.copy_(3 * torch.randn((rows, V), generator=g, device="cuda"))
    assert x.data_ptr() % 32 == 4 * front % 32
    targets = torch.randint(0, V, (rows, 3), generator=g, device="cuda", dtype=torch.int32)
    _check_logprobs(x, 1.0, targets, *_run_logprobs(x, 1.0, targets, k), "16 bytes off")
