"""moe_adamw: bit for bit against the same operations in numpy's fp32, and
within rounding of the definition in fp64."""
import numpy as np
import pytest
import torch

from _gpu_common import lib, need_gpu
from _train_common import DT, U, n64, u

pytestmark = pytest.mark.gpu

f32 = np.float32
M64 = 2 ** 64 - 1


def _mix64(x):
    x = (x + 0x9E3779B97F4A7C15) & M64
    x = ((x ^ (x >> 30)) * 0xBF58476D1CE4E5B9) & M64
    x = ((x ^ (x >> 27)) * 0x94D049BB133111EB) & M64
    return x ^ (x >> 31)


def _key(seed, k):
    return _mix64((seed + 0x9E3779B97F4A7C15 * k) & M64) >> 32


def _bits(n, key, first=0):
    """16 random bits of elements first .. first + n - 1."""
    i = np.arange(first, first + n, dtype=np.uint64)
    j = i >> np.uint64(1)
    h = (j.astype(np.uint32) ^ np.uint32(key)
         ^ ((j >> np.uint64(32)) * np.uint64(0x9E3779B9)).astype(np.uint32))
    h = (h ^ h >> np.uint32(16)) * np.uint32(0x85EBCA6B)
    h = (h ^ h >> np.uint32(13)) * np.uint32(0xC2B2AE35)
    h = h ^ h >> np.uint32(16)
    return np.where(i & np.uint64(1), h >> np.uint32(16), h & np.uint32(0xFFFF)).astype(np.int64)


def _values(codes, scale):
    """fp32 values of E4M3 codes (uint8) with a scale per 128."""
    v = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    with np.errstate(invalid="ignore"):
        return v * np.repeat(scale, 128)[:v.size]


def _blocks(x):
    return np.concatenate((x, np.zeros(-x.size % 128, f32))).reshape(-1, 128)


def _quotients(x, scale):
    b = _blocks(x)
    with np.errstate(all="ignore"):
        q = np.where(scale[:, None] == 0, f32(0), b / scale[:, None])
    return q.reshape(-1)[:x.size].astype(f32)


def _step32(t, c):
    """One step of one tensor in fp32, operation by operation; t is changed."""
    lr, b1, b2, eps, step, gs, seed = c
    g = t["g"].astype(f32) * f32(gs)
    if "ms" in t:
        m0, r0 = _values(t["m"], t["ms"]), _values(t["v"], t["vs"])
        v0 = r0 * r0
    else:
        m0, v0 = t["m"], t["v"]
    m = m0 * f32(b1) + g * f32(1.0 - b1)
    v = v0 * f32(b2) + (g * g) * f32(1.0 - b2)
    r = np.sqrt(v)
    size = f32(lr / (1.0 - b1 ** step))
    root = f32(1.0 / np.sqrt(1.0 - b2 ** step))
    p = t["master"] if t.get("master") is not None else t["p"].astype(f32)
    with np.errstate(all="ignore"):
        p = p * f32(1.0 - lr * t["wd"]) - m / (r * root + f32(eps)) * size
    assert p.dtype == m.dtype == v.dtype == f32
    if t.get("master") is not None:
        t["master"] = p
    t["p"] = p
    if "ms" not in t:
        t["m"], t["v"] = m, v
        return
    ms = np.abs(_blocks(m)).max(1) * f32(1.0 / 448.0)
    q = torch.from_numpy(_quotients(m, ms))
    t["m"] = q.to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    t["ms"] = ms
    rs = _blocks(r).max(1) * f32(1.0 / 448.0)
    q = _quotients(r, rs)
    w = _bits(r.size, t["key"])
    t20 = (q * f32(2.0 ** -120)).view(np.int32).astype(np.int64) + (w << 4) + 8
    code = t20 >> 20
    t["v"] = np.where((code == 0) & (r > 0), 1, code).astype(np.uint8)
    t["vs"] = rs


def _tensor(n, gen, param, grad, master, bits, wd, key, zero=False):
    """A tensor's state on the CPU; params are fp32 values of their type."""
    scale = torch.exp(torch.randn((n,), generator=gen))
    p = (torch.randn((n,), generator=gen) * 0.02).to(DT[param]).float()
    t = {"p": p.numpy(), "wd": wd, "key": key}
    t["g"] = (torch.randn((n,), generator=gen) * 1e-3 * scale).to(DT[grad]).float().numpy()
    if master:
        t["master"] = (p + torch.randn((n,), generator=gen) * 1e-5).numpy()
    m = 0.0 if zero else (torch.randn((n,), generator=gen) * 3e-4 * scale).numpy()
    r = 0.0 if zero else ((torch.rand((n,), generator=gen) + 0.1) * 1e-3 * scale).numpy()
    m, r = (np.broadcast_to(f32(v), (n,)).copy() if zero else v for v in (m, r))
    if bits == 32:
        t["m"], t["v"] = m, r * r
    else:
        for k, v in (("m", m), ("v", r)):
            t[k + "s"] = np.abs(_blocks(v)).max(1) * f32(1.0 / 448.0)
            q = torch.from_numpy(_quotients(v, t[k + "s"]))
            t[k] = q.to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    return t


GUARD = 64


def _device(t, param, grad):
    """Its buffers on the GPU, each followed by a guard."""
    def put(x, dtype, fill):
        x = torch.from_numpy(x).to(dtype)
        return torch.cat((x, torch.full((GUARD,), fill, dtype=dtype))).cuda()
    d = {"param": put(t["p"], DT[param], 5), "grad": put(t["g"], DT[grad], 5)}
    if t.get("master") is not None:
        d["master"] = put(t["master"], torch.float32, 5)
    state = torch.uint8 if "ms" in t else torch.float32
    d["exp_avg"], d["exp_avg_sq"] = put(t["m"], state, 5), put(t["v"], state, 5)
    if "ms" in t:  # the scales on any 4 bytes
        for name, x in (("exp_avg_scale", t["ms"]), ("exp_avg_sq_scale", t["vs"])):
            d[name] = torch.cat((torch.zeros(3, device="cuda"), put(x, torch.float32, 5)))[3:]
    d["n"], d["weight_decay"] = t["p"].size, t["wd"]
    return d


def _same(t, d, param):
    """Every value of the step, bit for bit, and the guards as they were."""
    for name, x in d.items():
        if isinstance(x, torch.Tensor):
            assert (x[-GUARD:].float() == 5).all(), name
    get = lambda k: d[k][:-GUARD].cpu()  # noqa: E731
    want = torch.from_numpy(t["p"]).to(DT[param])
    assert torch.equal(get("param"), want)
    if t.get("master") is not None:
        assert np.array_equal(get("master").numpy(), t["master"])
    assert np.array_equal(get("exp_avg").numpy(), t["m"])
    assert np.array_equal(get("exp_avg_sq").numpy(), t["v"])
    if "ms" in t:
        assert np.array_equal(get("exp_avg_scale").numpy(), t["ms"])
        assert np.array_equal(get("exp_avg_sq_scale").numpy(), t["vs"])


def _call(fgs, table, param, grad, bits, c, gs_dev, stream=None):
    code = {"bf16": fgs.MOE_BF16, "f32": fgs.MOE_F32}
    lr, b1, b2, eps, step, _, seed = c
    fgs.moe_adamw(table, code[param], code[grad], bits, lr, b1, b2, eps, step, gs_dev, seed, stream)


SIZES = [[1], [7], [128], [129, 1, 127], [4095, 4096, 4097, 0, 8193], [100_003],
         [3] * 300 + [260, 1000], [0, 0, 5, 0]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("param,grad,master", [("f32", "f32", False), ("f32", "bf16", False),
                                               ("bf16", "bf16", False), ("bf16", "bf16", True),
                                               ("bf16", "f32", True)])
def test_steps(sizes, bits, param, grad, master):
    """Two steps, the second from the first's states."""
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(len(sizes) + bits)
    seed = 2 ** 40 + 17
    ts = [_tensor(n, gen, param, grad, master, bits, 0.1 * (k % 2), _key(seed, k))
          for k, n in enumerate(sizes)]
    ds = [_device(t, param, grad) for t in ts]
    table = fgs.adamw_table(ds)
    gs = torch.tensor([0.37], device="cuda")
    for step in (1, 2):
        c = (1e-3, 0.9, 0.95, 1e-8, step, 0.37, seed)
        for t in ts:
            if t["p"].size:
                if param == "bf16" and not master:
                    t["p"] = torch.from_numpy(t["p"]).bfloat16().float().numpy()
                _step32(t, c)
        _call(fgs, table, param, grad, bits, c, gs)
        for t, d in zip(ts, ds):
            if t["p"].size:
                _same(t, d, param)


@pytest.mark.parametrize("bits", [8, 32])
def test_against_the_definition(bits):
    """Params, moments and scales within the roundings of fp32, from a state of
    zeros and over later steps, without a grad_scale."""
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(3)
    n = 5000
    t = _tensor(n, gen, "f32", "f32", False, bits, 0.1, 0, zero=True)
    d = _device(t, "f32", "f32")
    table = fgs.adamw_table([d])
    lr, b1, b2, eps = 1e-2, 0.9, 0.999, 1e-8
    for step in range(1, 6):
        g = torch.randn((n,), generator=gen) * 1e-3
        d["grad"][:n] = g.cuda()
        p, g = n64(d["param"][:n]), n64(g)
        if bits == 8:
            m, r = (_values(d[k][:-GUARD].cpu().numpy(), d[k + "_scale"][:-GUARD].cpu().numpy())
                    .astype(np.float64) for k in ("exp_avg", "exp_avg_sq"))
            v = r * r
        else:
            m, v = n64(d["exp_avg"][:n]), n64(d["exp_avg_sq"][:n])
        em = 4 * u * (b1 * np.abs(m) + (1 - b1) * np.abs(g))
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        up = m / (1 - b1 ** step) / (np.sqrt(v / (1 - b2 ** step)) + eps)
        want = p * (1 - lr * 0.1) - lr * up
        # v is within 6 roundings, its root 4, the divisor 7, and then m, the
        # quotient, its factor and its rounding, and p's two
        lim = lr * (np.abs(up) * 12 * u + em / (1 - b1 ** step)
                    / (np.sqrt(v / (1 - b2 ** step)) + eps))
        lim += 3 * u * (np.abs(p) + np.abs(lr * up))
        _call(fgs, table, "f32", "f32", bits, (lr, b1, b2, eps, step, 1.0, step), None)
        assert (np.abs(n64(d["param"][:n]) - want) <= lim).all()
        if bits == 32:
            assert (np.abs(n64(d["exp_avg"][:n]) - m) <= em).all()
            assert (np.abs(n64(d["exp_avg_sq"][:n]) - v) <= 6 * u * v).all()
            continue
        for name, x, least in (("exp_avg", m, 0.5), ("exp_avg_sq", np.sqrt(v), 1.0)):
            codes = d[name][:-GUARD].cpu().numpy()
            scale = d[name + "_scale"][:-GUARD].cpu().numpy()
            top = np.abs(_blocks(x.astype(f32))).max(1) / 448
            assert (np.abs(scale - top) <= 10 * u * top + em.max() / 448 * (name == "exp_avg")).all()
            # nearest is at most half a step of E4M3 off, at random a whole one;
            # a step is 2^-3 of the value's power of two, or 2^-9 scales
            s = np.repeat(scale, 128)[:n].astype(np.float64)
            one = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(x) / s, 1e-30))) - 3), 2.0 ** -9)
            off = np.abs(_values(codes, scale).astype(np.float64) - x)
            assert (off <= least * one * s * 1.0001 + em).all()


def test_second_moment_moves():
    """A root that should fall by 5% while its block's largest stays does so on
    average: rounding to nearest would hold it.  The mean of 127 x 512 elements'
    relative change: each of 100 roundings moves an element by at most a step,
    2^-3 of it, with a variance of at most a quarter of that squared, so the
    mean's deviation is below 10 x 2^-4 / 255 = 0.0025; six of them."""
    need_gpu()
    fgs = lib()
    n, steps, b2 = 128 * 512, 100, 0.999
    gen = torch.Generator().manual_seed(1)
    r = torch.rand((512, 128), generator=gen) * 0.2 + 0.1
    r[:, 0] = 1.0
    t = _tensor(n, gen, "f32", "f32", False, 8, 0.0, 0, zero=True)
    t["vs"] = np.full(512, f32(1.0 / 448.0))
    t["v"] = (r * 448).reshape(-1).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    t["g"] = np.zeros((512, 128), f32)
    t["g"][:, 0] = 1.0  # keeps the block's largest at 1
    t["g"] = t["g"].reshape(-1)
    d = _device(t, "f32", "f32")
    before = _values(t["v"], t["vs"]).reshape(512, 128)[:, 1:].astype(np.float64)
    table = fgs.adamw_table([d])
    for step in range(1, steps + 1):
        _call(fgs, table, "f32", "f32", 8, (0.0, 0.9, b2, 1e-8, step, 1.0, step), None)
    after = _values(d["exp_avg_sq"][:-GUARD].cpu().numpy(),
                    d["exp_avg_sq_scale"][:-GUARD].cpu().numpy()).reshape(512, 128)
    assert abs(after[:, 0] - 1).max() <= 1e-3
    change = (after[:, 1:] / before).mean()
    assert abs(change - b2 ** (steps / 2)) <= 0.015, change


def test_small_roots_keep_a_code():
    """A root far below its block's largest keeps code 1, so that the update of
    the next step, without a gradient, stays bounded."""
    need_gpu()
    fgs = lib()
    n = 256
    gen = torch.Generator().manual_seed(1)
    t = _tensor(n, gen, "f32", "f32", False, 8, 0.0, 0, zero=True)
    t["p"][:] = 0.0
    t["g"][:] = 1e-9
    t["g"][::128] = 1.0
    d = _device(t, "f32", "f32")
    table = fgs.adamw_table([d])
    _call(fgs, table, "f32", "f32", 8, (1e-3, 0.9, 0.999, 1e-12, 1, 1.0, 9), None)
    codes = d["exp_avg_sq"][:-GUARD].cpu().numpy()
    assert (codes[1:128] == 1).all() and (codes[129:] == 1).all()
    d["grad"][:n] = 0.0
    before = d["param"][:n].clone()
    _call(fgs, table, "f32", "f32", 8, (1e-3, 0.9, 0.999, 1e-12, 2, 1.0, 10), None)
    assert float((d["param"][:n] - before).abs().max()) <= 2e-3


def test_values_that_are_not_finite():
    """A NaN gradient spoils its element (32 bits) or its block of 128 (8 bits)
    and nothing else."""
    need_gpu()
    fgs = lib()
    for bits in (8, 32):
        for value in (float("nan"), float("inf")):
            gen = torch.Generator().manual_seed(6)
            t = _tensor(1000, gen, "f32", "f32", False, bits, 0.1, _key(3, 0))
            t["g"][300] = value  # in block 2
            d = _device(t, "f32", "f32")
            with np.errstate(all="ignore"):
                _step32(t, (1e-3, 0.9, 0.95, 1e-8, 3, 1.0, 3))
            _call(fgs, fgs.adamw_table([d]), "f32", "f32", bits, (1e-3, 0.9, 0.95, 1e-8, 3, 1.0, 3),
                  None)
            rest = np.r_[0:256, 384:1000] if bits == 8 else np.r_[0:300, 301:1000]
            p = d["param"][:1000].cpu().numpy()
            keep = np.r_[0:300, 301:1000]  # this step's params: the element alone
            assert np.array_equal(p[keep], t["p"][keep]) and np.isnan(p[300])
            for k, name in (("m", "exp_avg"), ("v", "exp_avg_sq")):
                assert np.array_equal(d[name][:1000].cpu().numpy()[rest], t[k][rest])
            if bits == 8:
                for name in ("exp_avg", "exp_avg_sq"):
                    v = _values(d[name][:1000].cpu().numpy(),
                                d[name + "_scale"][:8].cpu().numpy())
                    assert not np.isfinite(v[300]) and np.isfinite(v[rest]).all()


def test_grad_scale_is_read_on_the_device():
    """A captured step reads the value that its scalar holds at the replay."""
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(2)
    t = _tensor(3000, gen, "bf16", "bf16", True, 8, 0.1, _key(4, 0))
    d = _device(t, "bf16", "bf16")
    gs = torch.ones(1, device="cuda")
    table = fgs.adamw_table([d])
    _call(fgs, table, "bf16", "bf16", 8, (0.0, 0.0, 0.0, 1e-8, 1, 1.0, 4), gs)  # load the module
    for name, x in _device(t, "bf16", "bf16").items():
        if isinstance(x, torch.Tensor):
            d[name].copy_(x)
    c = (1e-3, 0.9, 0.95, 1e-8, 5, None, 4)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _call(fgs, table, "bf16", "bf16", 8, c, gs)
    for value in (0.5, 0.25):
        gs.fill_(value)
        graph.replay()
        torch.cuda.synchronize()
        _step32(t, c[:5] + (value, 4))
        _same(t, d, "bf16")


def test_large_tensor():
    """Element numbers past 2^32: their pairs' random bits, and their offsets."""
    need_gpu()
    fgs = lib()
    n = 2 ** 33 + 1000  # 8.6e9 elements: pairs past 2^32
    dev = dict(device="cuda")
    nb = -(-n // 128)
    d = {"param": torch.zeros(n, dtype=torch.bfloat16, **dev),
         "grad": torch.zeros(n, dtype=torch.bfloat16, **dev),
         "exp_avg": torch.zeros(n, dtype=torch.uint8, **dev),
         "exp_avg_sq": torch.zeros(n, dtype=torch.uint8, **dev),
         "exp_avg_scale": torch.zeros(nb, **dev), "exp_avg_sq_scale": torch.zeros(nb, **dev)}
    gen = torch.Generator().manual_seed(2)
    g = (torch.randn((1000,), generator=gen) * 1e-3).bfloat16()
    first = n - 1000
    assert first % 128 == 0
    d["grad"][first:] = g.cuda()
    _call(fgs, fgs.adamw_table([d]), "bf16", "bf16", 8, (1e-3, 0.9, 0.95, 1e-8, 1, 1.0, 77), None)
    t = {"p": np.zeros(1000, f32), "g": g.float().numpy(), "wd": 0.0, "m": np.zeros(1000, np.uint8),
         "v": np.zeros(1000, np.uint8), "ms": np.zeros(8, f32), "vs": np.zeros(8, f32),
         "key": _key(77, 0)}
    whole = globals()["_bits"]
    try:
        globals()["_bits"] = lambda k, key: whole(k, key, first)
        _step32(t, (1e-3, 0.9, 0.95, 1e-8, 1, 1.0, 77))
    finally:
        globals()["_bits"] = whole
    assert torch.equal(d["param"][first:].cpu(), torch.from_numpy(t["p"]).bfloat16())
    assert np.array_equal(d["exp_avg_sq"][first:].cpu().numpy(), t["v"])
    assert np.array_equal(d["exp_avg"][first:].cpu().numpy(), t["m"])
    assert not d["param"][:first].any()


def test_table_refuses_a_buffer_twice():
    need_gpu()
    fgs = lib()
    a, b, g, m, v, m2, v2 = (torch.zeros(256, device="cuda") for _ in range(7))
    one = dict(param=a, grad=g, exp_avg=m, exp_avg_sq=v)
    for two in (dict(param=a, grad=g, exp_avg=m2, exp_avg_sq=v2),
                dict(param=b, grad=g, exp_avg=m, exp_avg_sq=v2),
                dict(param=b, grad=a, exp_avg=m2, exp_avg_sq=v2),
                dict(param=g, grad=b, exp_avg=m2, exp_avg_sq=v2)):
        with pytest.raises(ValueError, match="already"):
            fgs.adamw_table([one, two])
    assert len(fgs.adamw_table([one, dict(param=b, grad=g, exp_avg=m2, exp_avg_sq=v2)])) == 2
