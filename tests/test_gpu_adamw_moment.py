"""moe_adamw's first moment in 8 bits: the codes that rounding to nearest would
give back, bit for bit against numpy's fp32, and weights that no gradient
reaches any more beside live ones of their block."""
import numpy as np
import pytest
import torch

from _gpu_common import lib, need_gpu
from test_gpu_adamw import (_bits, _blocks, _call, _device, _key, _quotients, _same, _step32,
                            _tensor, _values)

pytestmark = pytest.mark.gpu

f32 = np.float32


def _moment_bits(n, key):
    """16 random bits of the first moment's elements: those of the neighbour's root."""
    return _bits(n + n % 2, key).reshape(-1, 2)[:, ::-1].reshape(-1)[:n]


def _step(t, c):
    """_step32, with m's codes that nearest gives back rounded at random; how many
    there were, and how many of them changed."""
    old, b1 = t["m"].copy(), c[1]
    m = _values(old, t["ms"]) * f32(b1) + t["g"].astype(f32) * f32(c[5]) * f32(1.0 - b1)
    _step32(t, c)
    q = torch.from_numpy(_quotients(m, t["ms"])).clamp(-448, 448)  # codes saturate
    near = q.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    held = ((near ^ old) & 0x7F) == 0
    held &= (old & 0x7F) < (0x7F if b1 > 29 / 32 else 8)
    bits = (np.abs(_quotients(m, t["ms"])) * f32(2.0 ** -120)).view(np.int32).astype(np.int64)
    code = bits + (_moment_bits(m.size, t["key"]) << 4) + 8 >> 20
    code = np.minimum(code, 0x7E)
    t["m"] = np.where(held, code | (near & 0x80), near).astype(np.uint8)
    return int(held.sum()), int((t["m"] != near).sum())


@pytest.mark.parametrize("b1", [0.0, 0.9, 29 / 32, 0.95, 0.999])
@pytest.mark.parametrize("sizes", [[7], [128], [4095, 1, 8193], [40_003]],
                         ids=lambda s: f"{len(s)}x{max(s)}")
def test_held_codes(sizes, b1):
    """Two steps from codes of all magnitudes, most of them with gradients too small
    to move them, in one launch of few and one of many elements."""
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(len(sizes))
    seed = 991
    ts = [_tensor(n, gen, "f32", "f32", False, 8, 0.0, _key(seed, k)) for k, n in enumerate(sizes)]
    for t in ts:
        n = t["p"].size
        code = torch.randint(0, 0x7F, (n,), generator=gen) | torch.randint(0, 2, (n,), generator=gen) << 7
        small = torch.rand((n,), generator=gen) < 0.3
        code[small] = torch.randint(0, 9, (int(small.sum()),), generator=gen)
        t["m"] = code.to(torch.uint8).numpy()
        t["m"][::128] = 0x7E
        level = 10.0 ** (torch.rand((n,), generator=gen) * -8)
        t["g"] = (torch.randn((n,), generator=gen) * 1e-3 * level).numpy()
        t["g"][torch.rand((n,), generator=gen).numpy() < 0.5] = 0.0
        t["g"][::128] = np.abs(_values(t["m"], t["ms"]))[::128]  # the largest stays
    ds = [_device(t, "f32", "f32") for t in ts]
    table = fgs.adamw_table(ds)
    held = changed = 0
    for step in (1, 2):
        c = (1e-3, b1, 0.95, 1e-8, step, 0.75, seed)
        for t in ts:
            h, k = _step(t, c)
            held, changed = held + h, changed + k
        _call(fgs, table, "f32", "f32", 8, c, torch.tensor([0.75], device="cuda"))
        for t, d in zip(ts, ds):
            _same(t, d, "f32")
    if max(sizes) > 1000:
        assert held > 100 and (changed > 100 or b1 == 0.0)


@pytest.mark.parametrize("b1", [0.9, 0.95, 0.999])
def test_scales_of_a_few_bits(b1):
    """Blocks that no gradient has reached for so long that their scale is a few units
    of 2^-149, where a quotient can be up to half as much again as 448: codes stay
    finite, step after step, until all are 0."""
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(4)
    n = 128 * 200
    t = _tensor(n, gen, "f32", "f32", False, 8, 0.0, _key(8, 0))
    t["g"][:] = 0.0
    t["m"] = (torch.randint(0, 0x7F, (n,), generator=gen)
              | torch.randint(0, 2, (n,), generator=gen) << 7).to(torch.uint8).numpy()
    t["m"][::128] = 0x7E
    t["ms"] = np.concatenate((np.arange(1, 101, dtype=f32) * f32(2.0 ** -149),
                              f32(2.0) ** -np.arange(45, 145).astype(f32)))
    d = _device(t, "f32", "f32")
    table = fgs.adamw_table([d])
    for step in range(1, 41):
        c = (1e-3, b1, 0.95, 1e-8, step, 1.0, 8)
        _step(t, c)
        _call(fgs, table, "f32", "f32", 8, c, None)
        _same(t, d, "f32")
        assert ((t["m"] & 0x7F) < 0x7F).all() and np.isfinite(t["p"]).all()


@pytest.mark.parametrize("live", ["noise", "steady"])
@pytest.mark.parametrize("b1", [0.9, 0.95])
def test_weights_without_a_gradient_come_to_rest(b1, live):
    """Half of each block has no gradient after step 20.  Its moments fall by b1 a
    step: with b1 0.9 by at least a code while they are above code 7 (119 steps at
    most), then, with 0.95 from the start, by 1 - b1 of themselves on the average, as
    the random codes keep the mean.  So at step 400 a moment has less than 1e-3 of
    the least code on the average: 4 x 0.9^258 and 448 x 512 x 0.95^380 = 8e-4 of one.
    A step moves a weight by lr m / r, where r has at least the least code of its
    scale and m's scale is at most 1.3 times r's (|m| <= 1.17 r by the inequality of
    Cauchy and Schwarz for these factors): from there on by 1.3 x 8e-4 / 0.05 = 0.02 lr
    altogether, on the average of 2048 weights.  The chance that more than 1% of them
    still have a code then is that of ten times the mean number; each moves by at
    most some 20 lr, which bounds the mean by 0.2 lr.  Held by their codes they
    move by m / r in every one of the 600 steps: some tens of lr."""
    need_gpu()
    fgs = lib()
    n, steps, b2 = 4096, 1000, 0.95
    gen = torch.Generator(device="cuda").manual_seed(5)
    dead = torch.arange(n, device="cuda") % 2 == 1
    z = lambda k=n: torch.zeros(k, device="cuda")  # noqa: E731
    c = lambda: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    g, p8, p32 = z(), z(), z()
    t8 = fgs.adamw_table([dict(param=p8, grad=g, exp_avg=c(), exp_avg_sq=c(),
                               exp_avg_scale=z(n // 128), exp_avg_sq_scale=z(n // 128))])
    t32 = fgs.adamw_table([dict(param=p32, grad=g, exp_avg=z(), exp_avg_sq=z())])
    for step in range(1, steps + 1):
        if live == "noise":
            g.copy_(torch.randn((n,), generator=gen, device="cuda") + 1.0)
        else:
            g.fill_(1.0)
            g[dead] = 0.3 + 0.2 * torch.rand((n // 2,), generator=gen, device="cuda")
        if step > 20:
            g[dead] = 0.0
        for t, bits in ((t8, 8), (t32, 32)):
            _call(fgs, t, "f32", "f32", bits, (1.0, b1, b2, 1e-8, step, 1.0, step), None)
        if step == 400:
            from8, from32 = p8.clone(), p32.clone()
    off = ((p8 - from8) - (p32 - from32))[dead].abs()
    assert float(off.mean()) <= 0.2, (float(off.mean()), float(off.max()))


def test_untouched_blocks_stay_zero():
    """No gradient and no state: codes and scales stay 0, whatever beta1."""
    need_gpu()
    fgs = lib()
    for b1 in (0.9, 0.99):
        gen = torch.Generator().manual_seed(1)
        t = _tensor(1000, gen, "f32", "f32", False, 8, 0.1, _key(5, 0), zero=True)
        t["g"][:512] = 0.0
        d = _device(t, "f32", "f32")
        for step in (1, 2):
            c = (1e-3, b1, 0.95, 1e-8, step, 1.0, 5)
            _step(t, c)
            _call(fgs, fgs.adamw_table([d]), "f32", "f32", 8, c, None)
            _same(t, d, "f32")
        assert not t["m"][:512].any() and not t["ms"][:4].any()
        assert np.abs(_blocks(t["p"])).max() > 0


@pytest.mark.parametrize("bits", [8, 32])
def test_new_gradients(bits):
    """Gradients that a backward pass made anew: the step takes them, not those that
    the table was made with."""
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(9)
    ts = [_tensor(n, gen, "f32", "bf16", False, bits, 0.1, _key(3, k))
          for k, n in enumerate((1000, 7, 5000))]
    ds = [_device(t, "f32", "bf16") for t in ts]
    table = fgs.adamw_table(ds)
    for step in (1, 2):
        if step == 2:
            for t, d in zip(ts, ds):
                t["g"] = (torch.randn(t["g"].shape, generator=gen) * 1e-3).bfloat16().float().numpy()
                d["grad"] = torch.cat((torch.from_numpy(t["g"]).bfloat16(),
                                       torch.full((64,), 5.0, dtype=torch.bfloat16))).cuda()
            table.set_grads(d["grad"] for d in ds)
        c = (1e-3, 0.9, 0.95, 1e-8, step, 1.0, 3)
        for t in ts:
            (_step if bits == 8 else _step32)(t, c)
        _call(fgs, table, "f32", "bf16", bits, c, None)
        for t, d in zip(ts, ds):
            _same(t, d, "f32")
