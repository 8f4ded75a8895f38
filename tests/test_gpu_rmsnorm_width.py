"""moe_add_rmsnorm on the widest row that its arguments can name."""
import pytest
import torch

from _gpu_common import lib, need_gpu

pytestmark = pytest.mark.gpu


def test_a_row_of_2_to_the_31_columns():
    """A thread's step beyond the last of 2^31 - 1 columns passes 2^31."""
    need_gpu()
    fgs = lib()
    d = 2 ** 31 - 1
    x = torch.ones((d,), dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.tensor([2.0, -1.0, 0.0, 4.0, -2.0])
    w = torch.ones((d,), dtype=torch.bfloat16, device="cuda")
    w[-1] = 8.0
    y = torch.full((d + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    fgs.moe_add_rmsnorm(fgs.MOE_BF16, 1, d, x, None, w, 0.0, None, y)
    # the mean square is 1 within 2^-26
    assert (y[:d - 5] == 1.0).all()
    assert y[d - 5:].tolist() == [2.0, -1.0, 0.0, 4.0, -16.0] + [7.0] * 9
