"""moe_adamw's roots and quotients, each correctly rounded: every mantissa of a
root, and quotients of all magnitudes, against fp64.  An fp64 root or quotient of fp32
values rounds to the fp32 one: it has more than twice its digits and two."""
import pytest
import torch

from _gpu_common import lib, need_gpu

pytestmark = pytest.mark.gpu


def _step(fgs, m, v, eps=0.0, step=200, b=0.5):
    """-m' / (sqrt(v') + eps) of one step of p = 0 without a gradient, and m', v':
    beta 0.5, so that m' = m / 2 and v' = v / 2, with both corrections 1 by step 200."""
    z = lambda: torch.zeros_like(m)  # noqa: E731
    p, m, v = z(), m.clone(), v.clone()
    table = fgs.adamw_table([dict(param=p, grad=z(), exp_avg=m, exp_avg_sq=v)])
    fgs.moe_adamw(table, fgs.MOE_F32, fgs.MOE_F32, 32, 1.0, b, b, eps, step)
    return p, m, v


def _root(v):
    return v.double().sqrt().float()


@pytest.mark.parametrize("exponent", [-88, -40, 0, 60])
def test_every_root(exponent):
    """v' of every mantissa and both parities of the exponent, and m' the root that
    it should have: the quotient is 1 exactly where the kernel's root is that one."""
    need_gpu()
    fgs = lib()
    bits = torch.arange(1 << 24, device="cuda", dtype=torch.int32) + ((128 + exponent) << 23)
    v = bits.view(torch.float32)
    for half in (v[: 1 << 23], v[1 << 23:]):
        root = _root(half * 0.5)
        p, m, out = _step(fgs, root * 2, half)
        assert torch.equal(m, root) and torch.equal(out, half * 0.5)
        assert (p == -1.0).all()


@pytest.mark.parametrize("eps", [0.0, 1e-8, 1.0, 2.0 ** 50, 2.0 ** 70])
@pytest.mark.parametrize("low,high", [(-20, 20), (-64, 64), (-140, 120)])
def test_quotients(low, high, eps):
    """m' and v' of all mantissas, m' of magnitudes from 2^low to 2^high (subnormal
    ones and quotients beyond fp32's range among them), v' from 2^-100 to 2^70."""
    need_gpu()
    fgs = lib()
    n = 1 << 22
    gen = torch.Generator(device="cuda").manual_seed(high)
    rand = lambda: torch.rand((n,), generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    m = ((1 + rand()) * torch.exp2(torch.floor(low + rand() * (high - low)))).float()
    m = torch.where(rand() < 0.5, m, -m)
    m = torch.where(rand() < 0.02, torch.zeros_like(m), m)
    v = ((1 + rand()) * torch.exp2(torch.floor(-100 + rand() * 170))).float()
    # eight neighbours are computed together: of one magnitude, so that it decides
    each = torch.exp2(torch.floor(-100 + rand()[::8] * 170)).repeat_interleave(8)
    half = n // 2
    v[half:] = ((1 + rand()) * each).float()[half:]
    p, m1, v1 = _step(fgs, m, v, eps)
    assert torch.equal(m1, m * 0.5) and torch.equal(v1, v * 0.5)
    d = _root(v1) + torch.tensor(eps, device="cuda")  # one fp32 sum
    want = -(m1.double() / d.double()).float()
    assert torch.equal(p, want)
