"""The 8-bit output of moe_add_rmsnorm, code by code: RN_E4M3(v / scale)."""
import pytest
import torch

from _gpu_common import lib, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d", [(3, 128), (40, 4096), (320, 4096), (2, 20480), (1, 65536)])
def test_codes_are_the_rounded_quotients(T, d):
    """Rows whose quotients lie around the midpoints between codes: integers up
    to 448 times a factor of the row, with a 448 in every group."""
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(T + d)
    x = torch.randint(-447, 448, (T, d), generator=gen).float()
    x[:, ::128] = 448.0
    x *= torch.rand((T, 1), generator=gen) + 0.5
    y = torch.empty((T, d), device="cuda")
    y8 = torch.empty((T, d), dtype=torch.uint8, device="cuda")
    ys = torch.empty((T, d // 128), device="cuda")
    fgs.moe_add_rmsnorm(fgs.MOE_F32, T, d, x.cuda(), None, torch.ones(d, device="cuda"), 1e-6, None,
                        y, y8, ys)
    # y is v itself in fp32: the quotient correctly rounded to fp32, then to E4M3
    v = y.cpu().view(T, d // 128, 128)
    want = (v / ys.cpu()[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    diff = int((want.view(T, d) != y8.cpu()).sum())
    assert diff == 0, f"{diff} of {T * d} codes"


def test_a_group_whose_scale_is_zero():
    """max |v| / 448 below half of fp32's smallest value: scale and codes 0."""
    need_gpu()
    fgs = lib()
    x = torch.ones((2, 256))
    w = torch.ones(256)
    w[:128] = 2.0 ** -145
    y = torch.empty((2, 256), device="cuda")
    y8 = torch.empty((2, 256), dtype=torch.uint8, device="cuda")
    ys = torch.empty((2, 2), device="cuda")
    fgs.moe_add_rmsnorm(fgs.MOE_F32, 2, 256, x.cuda(), None, w.cuda(), 0.0, None, y, y8, ys)
    assert (y[:, :128] > 0).all()
    assert (ys[:, 0] == 0).all() and (y8[:, :128] == 0).all()
    assert (ys[:, 1] == y[:, 255] / 448.0).all() and (y8[:, 128:] == 0x7E).all()
