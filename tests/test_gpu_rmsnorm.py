"""moe_add_rmsnorm against a plain fp64 form."""
import numpy as np
import pytest
import torch

from _gpu_common import lib, need_gpu
from _int4_common import U_BF16, U_F32

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _run(T, d, dtype, residual, fp8, want_h=True, want_y=True, seed=0, x=None, eps=EPS):
    fgs = lib()
    gen = torch.Generator().manual_seed(seed + T + d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    if x is None:
        x = torch.randn((T, d), generator=gen) * torch.exp2(torch.rand((T, 1), generator=gen) * 6 - 3)
    a = x.to(dt)
    r = torch.randn((T, d), generator=gen).mul(3).to(dt) if residual else None
    w = (1 + 0.3 * torch.randn((d,), generator=gen)).to(dt)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    h = torch.full((T + 1, d), 9.0, dtype=dt, device="cuda") if want_h else None
    y = torch.full((T + 1, d), 9.0, dtype=dt, device="cuda") if want_y else None
    y8 = torch.full((T, d), 3, dtype=torch.uint8, device="cuda") if fp8 else None
    ys = torch.full((T, d // 128), 9.0, device="cuda") if fp8 else None
    fgs.moe_add_rmsnorm(fgs.MOE_BF16 if dtype == "bf16" else fgs.MOE_F32, T, d, cu(a), cu(r), cu(w),
                        eps, h, y, y8, ys)
    torch.cuda.synchronize()
    for t in (h, y):
        assert t is None or (t[T] == 9.0).all()  # nothing beyond row T
    f64 = lambda t: t.float().numpy().astype(np.float64)  # noqa: E731
    s = f64(a) + (f64(r) if residual else 0.0)
    with np.errstate(all="ignore"):
        v = s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * f64(w)
    return dict(a=a, r=r, w=w, h=h[:T].cpu() if want_h else None, y=y[:T].cpu() if want_y else None,
                y8=y8.cpu() if fp8 else None, ys=ys.cpu().numpy() if fp8 else None, s=s, v=v)


def _check(o, d, dtype):
    u = U_BF16 if dtype == "bf16" else U_F32
    s, v = o["s"], o["v"]
    # s is rounded to fp32 first, then to its type; v: the sum of d squares
    # loses at most 2^-24 of itself per addition along its longest chain (at
    # most d / 32 + 16 of them: a lane's values, then trees), half of which
    # survives the square root; s, the inverse root (2 ulp), and two products
    # are five further fp32 roundings
    tol_v = (0.5 * (d / 32 + 16) + 8) * U_F32
    if o["h"] is not None:
        assert (np.abs(o["h"].double().numpy() - s) <= (u + U_F32) * 1.001 * np.abs(s)).all()
    if o["y"] is not None:
        lim = (u + tol_v) * 1.001 * np.abs(v) + 1e-37
        assert (np.abs(o["y"].double().numpy() - v) <= lim).all()
    if o["y8"] is not None:
        m = np.abs(v).reshape(v.shape[0], -1, 128)
        scale = m.max(2) / 448.0
        assert (np.abs(o["ys"] - scale) <= (tol_v + 2 * U_F32) * 1.001 * scale).all()
        got = o["y8"].view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
        assert np.isfinite(got).all()
        q = v / np.where(scale > 0, np.repeat(scale, 1, 1), 1.0).repeat(128, axis=1)
        # E4M3 has 4 significant bits (half a unit is 2^-4 relative) down to
        # 2^-6, and a spacing of 2^-9 below
        lim = np.maximum(np.abs(q) * 2.0 ** -4, 2.0 ** -10) + np.abs(q) * (2 * tol_v + 4 * U_F32)
        assert (np.abs(got - q) <= lim).all()
        # the group's largest value has the largest code
        assert (np.abs(got).reshape(m.shape).max(2) == np.where(scale > 0, 448.0, 0.0)).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,fp8", [
    (1, 1, False), (3, 7, False), (2, 33, False), (5, 100, False), (1, 128, True), (9, 128, True),
    (4, 384, True), (1, 1000, False), (700, 640, True), (33, 1001, False), (17, 2048, True),
    (1, 7168, True), (160, 7168, True), (2, 8200, False), (3, 18432, True), (2, 40000, False),
    (1, 65664, True),
])
def test_norm(T, d, fp8, dtype, residual):
    need_gpu()
    _check(_run(T, d, dtype, residual, fp8), d, dtype)


@pytest.mark.parametrize("want_h,want_y,fp8", [(False, True, False), (True, False, True),
                                               (False, False, True), (False, True, True)])
def test_output_choices(want_h, want_y, fp8):
    need_gpu()
    full = _run(6, 1280, "bf16", True, True)
    o = _run(6, 1280, "bf16", True, fp8, want_h, want_y)
    _check(o, 1280, "bf16")
    for k in ("h", "y", "y8"):
        assert o[k] is None or torch.equal(o[k], full[k])


def test_zero_rows_and_groups():
    need_gpu()
    x = torch.randn((4, 512))
    x[1] = 0.0
    x[2, 128:256] = 0.0
    o = _run(4, 512, "bf16", False, True, x=x)
    _check(o, 512, "bf16")
    assert (o["y"][1] == 0).all() and (o["y8"][1].view(torch.float8_e4m3fn).float() == 0).all()
    assert (o["ys"][1] == 0).all() and o["ys"][2, 1] == 0
    # eps = 0 and a row of zeros: 0 / 0
    o = _run(4, 512, "f32", False, False, x=x, eps=0.0)
    assert torch.isnan(o["y"][1]).all() and torch.isfinite(o["y"][[0, 2, 3]]).all()


def test_nonfinite_rows_stay_in_their_rows():
    need_gpu()
    x = torch.randn((5, 384))
    clean = _run(5, 384, "bf16", False, True, x=x.clone())
    x[1, 130], x[3, 5] = float("nan"), float("inf")
    o = _run(5, 384, "bf16", False, True, x=x)
    for k in ("y", "y8"):
        assert torch.equal(o[k][[0, 2, 4]], clean[k][[0, 2, 4]])
    assert torch.isnan(o["y"][1]).all() and np.isnan(o["ys"][1]).all()
    assert (o["y8"][1] & 0x7F == 0x7F).all()
    # 1 / sqrt(inf) = 0: the finite values become 0, the infinity 0 * inf
    y3 = o["y"][3].float()
    assert torch.isnan(y3[5]) and (y3[[0, 200, 383]] == 0).all()


def test_large_values_and_magnitudes():
    """Squares that overflow nothing: rows of 1e18 in fp32."""
    need_gpu()
    x = torch.randn((3, 256)) * 1e17
    _check(_run(3, 256, "f32", False, True, x=x), 256, "f32")


def test_tiny_weights():
    """Groups whose 448 / max overflows fp32 still get the codes of v / scale."""
    need_gpu()
    fgs = lib()
    x = torch.randn((2, 256), generator=torch.Generator().manual_seed(4))
    w = torch.full((256,), 2.0 ** -122)
    w[128:] = 1.0
    y = torch.empty((2, 256), device="cuda")
    y8 = torch.empty((2, 256), dtype=torch.uint8, device="cuda")
    ys = torch.empty((2, 2), device="cuda")
    fgs.moe_add_rmsnorm(fgs.MOE_F32, 2, 256, x.cuda(), None, w.cuda(), EPS, None, y, y8, ys)
    v = y.double().cpu().view(2, 2, 128)
    s = ys.double().cpu()
    # the scale is rounded once, where fp32 is subnormal to a multiple of 2^-149
    assert ((s - v.abs().amax(2) / 448).abs() <= 2.0 ** -149 + s * 2 * U_F32).all()
    q = v / s[..., None]
    got = y8.cpu().view(torch.float8_e4m3fn).double().view(2, 2, 128)
    # one E4M3 rounding of the quotient, and saturation at 448
    lim = torch.maximum(q.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) + q.abs() * 8 * U_F32
    assert ((got - q.clamp(-448, 448)).abs() <= lim).all()


@pytest.mark.parametrize("which", ["h=x y=r", "h=r y=x", "y=x"])
@pytest.mark.parametrize("d", [100, 7168])
def test_in_place(which, d):
    need_gpu()
    fgs = lib()
    x = torch.randn((9, d), device="cuda").bfloat16()
    r = torch.randn((9, d), device="cuda").bfloat16()
    w = torch.rand((d,), device="cuda").bfloat16()
    h, y = torch.empty_like(x), torch.empty_like(x)
    fgs.moe_add_rmsnorm(fgs.MOE_BF16, 9, d, x, r, w, EPS, h, y)
    a, b = x.clone(), r.clone()
    ho, yo = {"h=x y=r": (a, b), "h=r y=x": (b, a), "y=x": (None, a)}[which]
    fgs.moe_add_rmsnorm(fgs.MOE_BF16, 9, d, a, b, w, EPS, ho, yo)
    assert torch.equal(yo, y) and (ho is None or torch.equal(ho, h))


def test_offsets_beyond_32_bits():
    need_gpu()
    T, d = 300100, 7168
    fgs = lib()
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, d), device="cuda").bfloat16()
    x[:-3] = 1.0
    w = torch.ones((d,), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    fgs.moe_add_rmsnorm(fgs.MOE_BF16, T, d, x, None, w, EPS, None, y)
    v = x[-3:].double()
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    # the bound of _check: one bf16 rounding and the fp32 sum of d squares
    lim = (U_BF16 + (0.5 * (d / 32 + 16) + 8) * U_F32) * 1.001
    assert ((y[-3:].double() - v).abs() <= lim * v.abs()).all()
    assert (y[0] == 1.0).all() and (y[T // 2] == 1.0).all()


def test_same_bits_every_run_and_on_a_side_stream():
    need_gpu()
    fgs = lib()
    x = torch.randn((50, 4096), device="cuda").bfloat16()
    w = torch.rand((4096,), device="cuda").bfloat16()
    outs = [torch.empty_like(x) for _ in range(4)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for i, y in enumerate(outs):
        fgs.moe_add_rmsnorm(fgs.MOE_BF16, 50, 4096, x, None, w, EPS, None, y,
                            stream=side if i % 2 else None)
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], y) for y in outs[1:])
