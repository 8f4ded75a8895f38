"""The persistent kernels for 4-bit weights where a block of threads has more
than one piece of work: units of the tensor-core kernels and tiles of the
streamed one, with counts that no number of SMs divides; rows as wide as the
layer's; the same bits on every run; banks of more than 2^32 bytes."""
import numpy as np
import pytest
import torch

from _gpu_common import lib, need_gpu, workspace
from _int4_common import bank, close, dequant64, dot_bound, swiglu64, values64
from test_gpu_int4 import _case, _gen, _rows

pytestmark = pytest.mark.gpu

FORMS = [(False, 32), (False, 128), (True, 32), (True, 128)]  # (E4M3 rows, columns of a scale)


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("rows8,group", FORMS)
@pytest.mark.parametrize("T,I,add", [(50, 384, True), (50, 128, False), (300, 384, False),
                                     (300, 128, True)])
def test_linear_of_many_units(T, I, add, rows8, group):
    """More than two and less than three rounds of units (128 outputs by up to
    64 or 128 tokens), the last block row short; an odd number of chunks."""
    need_gpu()
    fgs = lib()
    tiles = -(-T // 128)
    O = 128 * (-(-(2 * _sms() + 9) // tiles)) - 48
    gen = _gen(T + I + group)
    q, s = bank(gen, 1, O, I, group)
    x, xs, x64 = _rows(gen, T, I, rows8)
    W = fgs.pack_int4(fgs.MOE_PACK_PLAIN, q.cuda(), s.cuda())
    a = torch.randn((T, O), generator=gen).bfloat16().cuda() if add else None
    y = torch.full((T + 1, O), 7.0, dtype=torch.bfloat16, device="cuda")
    fgs.moe_linear_int4(T, I, O, group, x, xs, W, a, y)
    torch.cuda.synchronize()
    w = dequant64(q[0], s[0])
    ref, bound = x64 @ w.T, dot_bound(w, x64)
    if add:
        ref = ref + values64(a)
        bound = bound + 2.0 ** -23 * (np.abs(ref) + np.abs(values64(a)))
    close(y[:T], ref, bound)
    assert (y[T] == 7.0).all()


@pytest.mark.parametrize("rows8,group", FORMS)
@pytest.mark.parametrize("T,I,O", [(41, 7168, 144), (64, 7168, 80), (65, 7168, 272),
                                   (130, 7168, 144), (50, 18432, 16), (41, 32768, 48)])
def test_linear_of_wide_rows_on_the_tensor_cores(T, I, O, rows8, group):
    need_gpu()
    fgs = lib()
    gen = _gen(T + I + O + group)
    q, s = bank(gen, 1, O, I, group)
    x, xs, x64 = _rows(gen, T, I, rows8)
    W = fgs.pack_int4(fgs.MOE_PACK_PLAIN, q.cuda(), s.cuda())
    y = torch.empty((T, O), dtype=torch.bfloat16, device="cuda")
    fgs.moe_linear_int4(T, I, O, group, x, xs, W, None, y)
    w = dequant64(q[0], s[0])
    close(y, x64 @ w.T, dot_bound(w, x64))


@pytest.mark.parametrize("rows8,group", FORMS)
@pytest.mark.parametrize("T", [50, 300])
def test_linear_same_bits_every_run_on_the_tensor_cores(T, rows8, group):
    need_gpu()
    fgs = lib()
    gen = _gen(T)
    q, s = bank(gen, 1, 20000, 640, group)
    x, xs, _ = _rows(gen, T, 640, rows8)
    W = fgs.pack_int4(fgs.MOE_PACK_PLAIN, q.cuda(), s.cuda())
    outs = [torch.empty((T, 20000), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for i, y in enumerate(outs):
        fgs.moe_linear_int4(T, 640, 20000, group, x, xs, W, None, y,
                            stream=side if i % 2 else None)
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], y) for y in outs[1:])


def _sizes_idx(sizes, seed):
    """One expert a token, sizes[e] tokens on expert e, shuffled."""
    idx = np.concatenate([np.full(n, e) for e, n in enumerate(sizes)])
    np.random.default_rng(seed).shuffle(idx)
    return idx[:, None]


@pytest.mark.parametrize("rows8,group", FORMS)
def test_experts_of_many_streamed_tiles(rows8, group):
    """Experts of 0 to 40 rows, several tiles of eight rows for a CTA: a
    beginning of a tile counts as 128 records and a tile here has 32 or 48."""
    need_gpu()
    sizes = [(7 * e) % 41 for e in range(300)]
    idx = _sizes_idx(sizes, 1)
    _case(len(idx), 256, 128, len(sizes), 1, 0, 0, 0, group, idx, rows8, 21)


@pytest.mark.parametrize("rows8,group", FORMS)
def test_experts_of_many_units(rows8, group):
    """Experts of 41 to 130 rows beside some with fewer, over more than two
    rounds of units in the gate/up pass, and a wider shared expert."""
    need_gpu()
    sizes = [41 + (29 * e) % 90 for e in range(44)] + [3, 0, 17, 40, 1]
    idx = _sizes_idx(sizes, 2)
    _case(len(idx), 384, 512, len(sizes), 1, 1, 640, 0, group, idx, rows8, 22)


@pytest.mark.parametrize("rows8", [False, True])
def test_experts_of_9_to_40_rows(rows8):
    """The rows an expert has when a few hundred tokens are decoded together."""
    need_gpu()
    g = np.random.default_rng(5)
    idx = np.stack([g.choice(96, 8, replace=False) for _ in range(256)])
    n = np.bincount(idx.ravel())
    assert n.min() >= 9 and n.max() <= 40
    _case(256, 512, 256, 96, 8, 1, 256, 0, 32, idx, rows8, 23)


@pytest.mark.parametrize("rows8,group", FORMS)
def test_experts_same_bits_every_run_on_the_tensor_cores(rows8, group):
    need_gpu()
    idx = _sizes_idx([60, 129, 41, 8, 200], 3)
    a = _case(len(idx), 256, 128, 5, 1, 1, 256, 0, group, idx, rows8, 24)
    b = _case(len(idx), 256, 128, 5, 1, 1, 256, 0, group, idx, rows8, 24)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("rows8,group", FORMS)
def test_experts_of_many_rows_in_banks_beyond_4_gib(rows8, group):
    """The last experts of a bank of more than 2^32 bytes, on the tensor cores."""
    need_gpu()
    fgs = lib()
    E, d, F, T = 304, 7168, 2048, 100
    g = torch.Generator(device="cuda").manual_seed(2)
    banks = {}
    for k, rows, cols in (("gu", 2 * F, d), ("dn", d, F)):
        q = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device="cuda",
                          dtype=torch.uint8)
        s = (torch.rand((E, rows, cols // group), generator=g, device="cuda") * 0.01).bfloat16()
        banks[k] = (q[-2:].clone(), s[-2:].clone(), fgs.pack_int4(0 if k == "gu" else 1, q, s))
        del q, s
    assert banks["gu"][2].numel() > 1 << 32
    cfg = fgs.config(d_model=d, d_ff=F, E_routed=E, K=1, weight_layout=3 if group == 32 else 4)
    ws, nws = workspace(cfg, T)
    x, xs, x64 = _rows(_gen(3), T, d, rows8)
    perm = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).contiguous()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E - 1:] = torch.tensor([55, T], dtype=torch.int32, device="cuda")
    Y = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    if rows8:
        fgs.moe_grouped_swiglu_fp8_rows(cfg, T, x, xs, off, perm, None, banks["gu"][2],
                                        banks["dn"][2], None, None, None, None, Y, None, ws, nws)
    else:
        fgs.moe_grouped_swiglu(cfg, T, x, off, perm, None, banks["gu"][2], banks["dn"][2], None,
                               None, None, Y, None, ws, nws)
    for e, rows in ((0, [0, 31, 54]), (1, [55, 99])):
        y, b = swiglu64(x64[[T - 1 - r for r in rows]], dequant64(*[t[e] for t in banks["gu"][:2]]),
                        dequant64(*[t[e] for t in banks["dn"][:2]]))
        close(Y[rows], y, b)
