"""The layer norm and its gradient where the first values of a row are unlike the
rest: many rows take their sums about the mean of those.  The bounds are those of
sums about the row's mean: the differences' roundings, half an ulp of |s - mu|
each, are in them."""
import numpy as np
import pytest
import torch

from _gpu_common import lib, need_gpu
from _train_common import U, close, n64, norm64, norm_backward64, u
from test_gpu_layernorm import EPS, _backward, _check_forward, _forward, _inputs

pytestmark = pytest.mark.gpu


def _rows(T, d, dtype):
    """Rows of normal values whose first 32 lie 0 to 10000 deviations off, all to
    one side, on both sides, or one of them alone; some with a mean of as many."""
    x, r, w, b, dy, dh = _inputs(T, d, dtype, seed=3, offset=0.0)
    gen = torch.Generator().manual_seed(T + d)
    x = torch.randn((T, d), generator=gen)
    far = torch.tensor([0.0, 1.0, 5.0, 10.0, 30.0, 100.0, 1000.0, 10000.0])
    t = torch.arange(T)
    k = far[t % 8] * torch.where(t // 8 % 2 == 0, 1.0, -1.0)
    how = t // 16 % 5
    x[:, :32] += torch.where(how == 0, k, 0.0)[:, None]
    x[:, 1:32:2] += torch.where(how == 1, k, 0.0)[:, None]
    x[:, 5] += torch.where(how == 2, k, 0.0)
    x += torch.where(how == 3, k, 0.0)[:, None]
    x[:, 32:] += torch.where(how == 4, k, 0.0)[:, None]
    return x.to(w.dtype), r.mul(0.1).to(w.dtype), w, b, dy, dh


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,d,dtype", [(701, 7001, "bf16"), (400, 577, "bf16"), (500, 1001, "f32"),
                                       (399, 7001, "f32"), (333, 8183, "f32"), (1300, 1001, "bf16")])
def test_forward_odd_rows(T, d, dtype, residual):
    need_gpu()
    fgs = lib()
    x, r, w, b, _, _ = _rows(T, d, dtype)
    r = r if residual else None
    h, y = _forward(fgs, dtype, x, r, w, b)
    _check_forward(dtype, x, r, w, b, h, y)
    # the same in place
    xd = x.cuda()
    out = torch.empty_like(xd)
    fgs.moe_add_layernorm(fgs.MOE_BF16 if dtype == "bf16" else fgs.MOE_F32, T, d, xd,
                          None if r is None else r.cuda(), w.cuda(), b.cuda(), 1e-6, xd, out)
    assert torch.equal(xd.cpu(), h) and torch.equal(out.cpu(), y)


@pytest.mark.parametrize("others", [0, 1, 3])
@pytest.mark.parametrize("T,d", [(2485, 1042), (3100, 577), (400, 7001)])
def test_forward_one_value_far_off(T, d, others):
    """One of the first values 1000 or 10000 deviations off, and as far off on either
    side some behind: the rest of the row lies about a deviation off the pivot, and its
    sum's roundings are not to be those of such values."""
    need_gpu()
    fgs = lib()
    for k in (1e3, 1e4):
        _, _, w, b, _, _ = _inputs(1, d, "f32")
        x = torch.randn((T, d), generator=torch.Generator().manual_seed(4))
        x[:, 5] += k
        for j in range(others):
            x[:, 200 + 100 * j] += k if j % 2 else -k
        _check_forward("f32", x, None, w, b, *_forward(fgs, "f32", x, None, w, b))


def _check(dtype, x, r, w, dy, dh, got):
    """As _check_backward, but dx ends in three roundings of its size where dh makes
    it up: of dh - r mean g, of the sum of that and r u c, and of the sum of that
    and r g.  norm_backward64 counts one, and close the last; the first, at most
    u (|dh| + r |mean g|), is added here."""
    X, R, W, DY, DH = (None if t is None else n64(t) for t in (x, r, w, dy, dh))
    want, lim = norm_backward64("layer", X, R, W, EPS, DY, DH)
    rs = norm64("layer", X, R, W, None, EPS)[2]
    more = u * (np.abs(DH) + rs * np.abs((DY * W).mean(1, keepdims=True))) * 1.01
    close(got["dx"], want[0], lim[0] + more, U[dtype])
    close(got["dw"], want[1], lim[1], u)
    close(got["db"], want[2], lim[2], u)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,d,dtype", [(1701, 7168, "bf16"), (3100, 520, "bf16"), (1601, 4104, "bf16"),
                                       (1101, 1000, "f32"), (1100, 7168, "f32"), (1101, 512, "f32"),
                                       (3101, 1001, "bf16"), (1603, 7001, "bf16"), (3101, 999, "f32"),
                                       (400, 8003, "f32")])
def test_backward(T, d, dtype, residual):
    need_gpu()
    fgs = lib()
    x, r, w, _, dy, dh = _rows(T, d, dtype)
    r = r if residual else None
    got = _backward(fgs, "layer", dtype, x, r, w, dy, dh)
    _check(dtype, x, r, w, dy, dh, got)
    t = x.cuda()
    again = _backward(fgs, "layer", dtype, t, r, w, dy, dh, dx=t)
    for name in got:
        assert torch.equal(got[name], again[name])
