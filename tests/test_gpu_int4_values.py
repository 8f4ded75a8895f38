"""Products with 4-bit weights at values off the ordinary: infinities and NaN
in rows, scales far apart within a row, scales near the ends of fp32's range,
and large values beside ordinary ones, on both sides of the limit between the
streamed and the tensor-core kernels (40 rows of a group)."""
import numpy as np
import pytest
import torch

from _gpu_common import lib, need_gpu
from _int4_common import bank, close, dequant64, dot_bound
from test_gpu_int4 import _gen, _rows

pytestmark = pytest.mark.gpu

# one token, the last streamed count, the first of the tensor cores, and both
# sides of a 64- and of a 128-token unit
TOKENS = [3, 40, 41, 64, 65, 130]


def _linear(x, xs, q, s, group):
    fgs = lib()
    W = fgs.pack_int4(fgs.MOE_PACK_PLAIN, q.cuda(), s.cuda())
    O, I = q.shape[1], 2 * q.shape[2]
    y = torch.full((x.shape[0], O), 7.0, dtype=torch.bfloat16, device="cuda")
    fgs.moe_linear_int4(x.shape[0], I, O, group, x, xs, W, None, y)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T", TOKENS)
def test_nonfinite_bf16_rows(T, group):
    """An infinity or a NaN of x gives what the definition gives (an infinity
    of the weight's sign, NaN at a zero weight), in its row alone."""
    need_gpu()
    gen = _gen(T + group)
    q, s = bank(gen, 1, 272, 384, group)
    x, _, x64 = _rows(gen, T, 384, False)
    clean = _linear(x, None, q, s, group)
    values = {0: {200: np.inf}, 1: {7: -np.inf, 130: -np.inf}, T - 1: {383: np.nan}}
    for row, at in values.items():
        for col, v in at.items():
            x[row, col], x64[row, col] = v, v
    y = _linear(x, None, q, s, group)
    w = dequant64(q[0], s[0])
    with np.errstate(invalid="ignore"):
        ref = x64[sorted(values)] @ w.T
    assert np.isinf(ref).any() and np.isnan(ref).any()
    got = y[sorted(values)].double().cpu().numpy()
    np.testing.assert_array_equal(got, ref)  # infinities with their signs, and NaN
    keep = [t for t in range(T) if t not in values]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T", TOKENS)
def test_nan_codes_stay_in_their_rows(T, group):
    need_gpu()
    gen = _gen(T + group)
    q, s = bank(gen, 1, 272, 384, group)
    x, xs, _ = _rows(gen, T, 384, True)
    clean = _linear(x, xs, q, s, group)
    x[0, 5], x[T - 1, 383] = 0x7F, 0xFF
    y = _linear(x, xs, q, s, group)
    assert torch.isnan(y[[0, T - 1]]).all()
    assert torch.equal(y[1:T - 1], clean[1:T - 1])


@pytest.mark.parametrize("rows8", [False, True])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("apart", [20, 27, 60])
@pytest.mark.parametrize("T", [5, 48, 100])
def test_scales_far_apart(T, apart, group, rows8):
    """A row's scales 2^apart from one group of columns to the next, with rows
    of x that are zero where the scales are large: what is left has to be right
    by itself."""
    need_gpu()
    gen = _gen(T * 100 + apart + group)
    q, s = bank(gen, 1, 144, 512, group)
    # every fourth group of a row large, from another one on in every row
    large = (torch.arange(512 // group) + torch.arange(144)[:, None]) % 4 == 0
    s[0] = torch.where(large, s[0].float(), s[0].float() * 2.0 ** -apart).bfloat16()
    x, xs, x64 = _rows(gen, T, 512, rows8)
    zero = torch.arange(512) // group % 4  # row t of x is zero in groups t mod 4
    mask = zero == torch.arange(T)[:, None] % 4
    x[mask.cuda()] = 0
    x64[mask.numpy()] = 0
    w = dequant64(q[0], s[0])
    close(_linear(x, xs, q, s, group), x64 @ w.T, dot_bound(w, x64))


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("x_exp,s_exp", [(121, -100), (-110, 127), (-100, -18), (100, -110)])
@pytest.mark.parametrize("T", [5, 48, 100])
def test_scales_near_the_ends_of_the_range(T, x_exp, s_exp, group):
    """Scales whose products with the outputs' other factors leave fp32's range
    although the outputs are far inside it."""
    need_gpu()
    gen = _gen(T + x_exp + s_exp + 300)
    q, s = bank(gen, 1, 144, 512, group)
    s = (s.double() * 2.0 ** s_exp).bfloat16()
    x, xs, x64 = _rows(gen, T, 512, True)
    xs, x64 = xs * 2.0 ** x_exp, x64 * 2.0 ** x_exp
    assert torch.isfinite(xs).all() and torch.isfinite(s).all()
    w = dequant64(q[0], s[0])
    close(_linear(x, xs, q, s, group), x64 @ w.T, dot_bound(w, x64))


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T", [5, 40, 48, 100])
def test_large_values_beside_ordinary_ones(T, group):
    """bf16 rows with values up to 2^30 times the smallest ones in columns whose
    weights are zero: the others' products are right by themselves."""
    need_gpu()
    gen = _gen(T + group)
    q, s = bank(gen, 1, 144, 512, group)
    q[:, :, ::32] = 0x88  # columns 0 and 1 of every 64: code 8, weight 0
    sign = torch.randint(0, 2, (T, 512), generator=gen) * 2 - 1
    x = (torch.rand((T, 512), generator=gen) * 3 + 1) * sign
    x.view(T, 8, 64)[:, :, :2] *= 2.0 ** 28
    x = x.bfloat16()
    w, x64 = dequant64(q[0], s[0]), x.double().numpy()
    close(_linear(x.cuda(), None, q, s, group), x64 @ w.T, dot_bound(w, x64))
