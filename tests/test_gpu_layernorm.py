"""moe_add_layernorm and moe_norm_backward against plain fp64 forms."""
import numpy as np
import pytest
import torch

from _gpu_common import lib, need_gpu
from _train_common import DT, U, chain, close, n64, norm64, norm_backward64, norm_errors, u

pytestmark = pytest.mark.gpu

EPS = 1e-6
KIND = {"rms": 0, "layer": 1}


def _inputs(T, d, dtype, seed=0, offset=0.5):
    gen = torch.Generator().manual_seed(seed + 131 * T + d)
    dt = DT[dtype]
    rows = torch.exp2(torch.rand((T, 1), generator=gen) * 6 - 3)
    x = ((torch.randn((T, d), generator=gen) + offset) * rows).to(dt)
    r = torch.randn((T, d), generator=gen).mul(3).to(dt)
    w = (1 + 0.3 * torch.randn((d,), generator=gen)).to(dt)
    b = torch.randn((d,), generator=gen).to(dt)
    dy, dh = (torch.randn((T, d), generator=gen).to(dt) for _ in range(2))
    return x, r, w, b, dy, dh


def _code(fgs, dtype):
    return fgs.MOE_BF16 if dtype == "bf16" else fgs.MOE_F32


def _forward(fgs, dtype, x, r, w, b, eps=EPS, h=True):
    T, d = x.shape
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    h = torch.full((T + 1, d), 9.0, dtype=x.dtype, device="cuda") if h else None
    y = torch.full((T + 1, d), 9.0, dtype=x.dtype, device="cuda")
    fgs.moe_add_layernorm(_code(fgs, dtype), T, d, cu(x), cu(r), cu(w), cu(b), eps, h, y)
    for t in (h, y):
        assert t is None or (t[T] == 9.0).all()  # nothing beyond row T
    return None if h is None else h[:T].cpu(), y[:T].cpu()


def _check_forward(dtype, x, r, w, b, h, y, eps=EPS):
    f = lambda t: None if t is None else n64(t)  # noqa: E731
    s, v, rs, want = norm64("layer", f(x), f(r), f(w), f(b), eps)
    if h is not None:
        close(h, s, u * np.abs(s), U[dtype])
    ev, _ = norm_errors("layer", s, rs, x.shape[1], eps)
    lim = np.abs(f(w)) * (ev + 2 * u * np.abs(v)) + u * np.abs(want)
    close(y, want, lim, U[dtype])


# a warp a row, a block a row with one, two or four pieces a thread, rows that
# are read again; widths of whole 16-byte pieces and others
WIDTHS = [1, 2, 3, 8, 31, 64, 128, 250, 256, 264, 1000, 1001, 1024, 1032, 1536, 2000, 4097, 7168,
          7170, 8192, 8200, 16384, 16385, 33001]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_forward_widths(d, dtype):
    need_gpu()
    fgs = lib()
    x, r, w, b, _, _ = _inputs(5, d, dtype)
    _check_forward(dtype, x, r, w, b, *_forward(fgs, dtype, x, r, w, b))


@pytest.mark.parametrize("residual,bias,h", [(False, False, False), (False, True, True),
                                             (True, False, True), (True, True, False)])
@pytest.mark.parametrize("T,d,dtype", [(1, 7168, "bf16"), (400, 7168, "bf16"), (333, 1000, "f32"),
                                       (9, 128, "bf16"), (700, 3584, "f32"), (1000, 520, "bf16")])
def test_forward(T, d, dtype, residual, bias, h):
    need_gpu()
    fgs = lib()
    x, r, w, b, _, _ = _inputs(T, d, dtype)
    r, b = r if residual else None, b if bias else None
    _check_forward(dtype, x, r, w, b, *_forward(fgs, dtype, x, r, w, b, h=h))


@pytest.mark.parametrize("T,d,dtype", [(1601, 257, "bf16"), (1600, 262, "bf16"), (1001, 1001, "bf16"),
                                       (700, 1002, "bf16"), (401, 1001, "f32"), (5001, 258, "f32"),
                                       (603, 7001, "bf16"), (305, 8175, "bf16"), (400, 8177, "bf16"),
                                       (333, 8183, "f32"), (20001, 300, "bf16")])
def test_forward_many_odd_rows(T, d, dtype):
    """Rows that begin inside a 16-byte chunk, in every place of it, beside rows of
    infinities and NaN; the last row ends where the tensors do."""
    need_gpu()
    fgs = lib()
    x, r, w, b, _, _ = _inputs(T, d, dtype)
    h, y = _forward(fgs, dtype, x, r, w, b)
    _check_forward(dtype, x, r, w, b, h, y)
    none = _forward(fgs, dtype, x, None, w, None, h=False)[1]
    _check_forward(dtype, x, None, w, None, None, none)
    xd, rd = x.cuda(), r.cuda()
    fgs.moe_add_layernorm(_code(fgs, dtype), T, d, xd, rd, w.cuda(), b.cuda(), EPS, xd, rd)
    assert torch.equal(xd.cpu(), h) and torch.equal(rd.cpu(), y)
    for row in (0, 200, T - 1):
        bad, keep = x.clone(), torch.arange(T) != row
        bad[row] = float("nan") if row else float("inf")
        h1, y1 = _forward(fgs, dtype, bad, r, w, b)
        assert torch.equal(h1[keep], h[keep]) and torch.equal(y1[keep], y[keep])
        assert y1[row].isnan().all()


@pytest.mark.parametrize("T,d,dtype", [(304, 7001, "bf16"), (400, 5555, "f32"), (2432, 1001, "bf16")])
def test_forward_odd_rows_in_place_repeats(T, d, dtype):
    """h in place of an input whose rows' first values every warp reads: the same
    bits each time."""
    need_gpu()
    fgs = lib()
    x, r, w, b, _, _ = (t.cuda() for t in _inputs(T, d, dtype))
    h, y = torch.empty_like(x), torch.empty_like(x)
    fgs.moe_add_layernorm(_code(fgs, dtype), T, d, x, r, w, b, EPS, h, y)
    for _ in range(10):
        for first in (True, False):
            xd, rd, out = x.clone(), r.clone(), torch.empty_like(x)
            at = xd if first else rd
            fgs.moe_add_layernorm(_code(fgs, dtype), T, d, xd, rd, w, b, EPS, at, out)
            assert torch.equal(at, h) and torch.equal(out, y)


@pytest.mark.parametrize("d", [64, 1000, 7168, 20000])
def test_forward_large_mean(d):
    """Rows whose mean is a thousand times their spread: sums of squares would
    lose the variance."""
    need_gpu()
    fgs = lib()
    x, _, w, b, _, _ = _inputs(7, d, "f32", offset=1000.0)
    _check_forward("f32", x, None, w, b, *_forward(fgs, "f32", x, None, w, b))


def test_forward_values():
    """Constant rows, eps 0, infinities and NaN: what the definition gives, in
    the row alone."""
    need_gpu()
    fgs = lib()
    d = 512
    x = torch.randn((6, d), generator=torch.Generator().manual_seed(1))
    x[0] = 3.0
    x[1] = 0.0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    w, b = torch.ones(d), torch.full((d,), 0.25)
    _, y = _forward(fgs, "f32", x, None, w, b)
    assert (y[0] == 0.25).all() and (y[1] == 0.25).all()
    assert y[2].isnan().all() and y[3].isnan().all()
    _check_forward("f32", x[4:], None, w, b, None, y[4:])
    _, y = _forward(fgs, "f32", x, None, w, b, eps=0.0)
    assert y[1].isnan().all()  # 0 / 0
    _check_forward("f32", x[4:], None, w, b, None, y[4:], eps=0.0)


@pytest.mark.parametrize("d", [100, 1000, 7168, 33001])
def test_forward_in_place(d):
    need_gpu()
    fgs = lib()
    x, r, w, b, _, _ = _inputs(5, d, "bf16")
    h, y = _forward(fgs, "bf16", x, r, w, b)
    for first in (True, False):
        xd, rd = x.cuda(), r.cuda()
        a, c = (xd, rd) if first else (rd, xd)
        fgs.moe_add_layernorm(fgs.MOE_BF16, 5, d, xd, rd, w.cuda(), b.cuda(), EPS, a, c)
        assert torch.equal(a.cpu(), h) and torch.equal(c.cpu(), y)


# ------------------------------------------------------------------ backward
def _backward(fgs, kind, dtype, x, r, w, dy, dh, want=("dx", "dw", "db"), eps=EPS, dx=None):
    T, d = x.shape
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    if dx is None and "dx" in want:
        dx = torch.full((T + 1, d), 9.0, dtype=x.dtype, device="cuda")
    dw = torch.full((d + 1,), 9.0, device="cuda") if "dw" in want else None
    db = torch.full((d + 1,), 9.0, device="cuda") if "db" in want and kind == "layer" else None
    n = fgs.moe_norm_backward_workspace_size(T, d)
    ws = torch.full((n + 256,), 0x5a, dtype=torch.uint8, device="cuda")
    sums = dw is not None or db is not None
    fgs.moe_norm_backward(KIND[kind], _code(fgs, dtype), T, d, cu(x), cu(r), cu(w), eps, cu(dy),
                          cu(dh), dx, dw, db, ws if sums else None, n if sums else 0)
    assert (ws[n:] == 0x5a).all()  # nothing beyond the workspace
    for t in (dw, db):
        assert t is None or float(t[d]) == 9.0
    if dx is not None and dx.shape[0] == T + 1:
        assert (dx[T] == 9.0).all()
        dx = dx[:T]
    return {"dx": dx, "dw": None if dw is None else dw[:d], "db": None if db is None else db[:d]}


def _check_backward(kind, dtype, x, r, w, dy, dh, got, eps=EPS):
    f = lambda t: None if t is None else n64(t)  # noqa: E731
    want, lim = norm_backward64(kind, f(x), f(r), f(w), eps, f(dy), f(dh))
    for name, a, b, rounding in zip(("dx", "dw", "db"), want, lim, (U[dtype], u, u)):
        if got[name] is not None:
            close(got[name], a, b, rounding)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_backward_widths(d, dtype, kind):
    need_gpu()
    fgs = lib()
    x, _, w, _, dy, dh = _inputs(5, d, dtype)
    _check_backward(kind, dtype, x, None, w, dy, dh,
                    _backward(fgs, kind, dtype, x, None, w, dy, dh))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d,dtype", [(1, 7168, "bf16"), (2, 40, "f32"), (303, 1000, "f32"),
                                       (305, 512, "bf16"), (700, 7168, "bf16"), (3000, 256, "bf16"),
                                       (2433, 60, "f32"), (650, 2048, "f32"), (100, 8201, "bf16"),
                                       (1100, 77, "bf16")])
def test_backward_rows(T, d, dtype, kind):
    """More rows than blocks, fewer, and a last block with fewer than the others."""
    need_gpu()
    fgs = lib()
    x, r, w, _, dy, dh = _inputs(T, d, dtype)
    _check_backward(kind, dtype, x, r, w, dy, dh, _backward(fgs, kind, dtype, x, r, w, dy, dh))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("residual,dh", [(False, True), (True, True), (False, False), (True, False)])
@pytest.mark.parametrize("T,d,dtype", [(1025, 264, "bf16"), (1027, 520, "f32"), (1029, 1032, "bf16"),
                                       (2501, 1000, "f32"), (2455, 136, "bf16"), (1433, 2048, "bf16"),
                                       (1100, 4096, "f32"), (2467, 7168, "bf16"),
                                       (1201, 8192, "bf16"), (1031, 7172, "f32"),
                                       (1025, 9000, "f32"), (1300, 8200, "bf16")])
def test_backward_many_rows(T, d, dtype, residual, dh, kind):
    """Rows that a block takes one after the other, or two at a time with one
    left over; all outputs, then dx in place of the gradient."""
    need_gpu()
    fgs = lib()
    x, r, w, _, dy, g = _inputs(T, d, dtype)
    r, g = r if residual else None, g if dh else None
    got = _backward(fgs, kind, dtype, x, r, w, dy, g)
    _check_backward(kind, dtype, x, r, w, dy, g, got)
    t = dy.cuda()
    again = _backward(fgs, kind, dtype, x, r, w, t, g, dx=t)
    for name in got:
        assert got[name] is None or torch.equal(got[name], again[name])


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d", [96, 1000, 7168, 20000])
@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dw", "db"), ("dx", "dw"), ("db",)])
def test_backward_some_outputs(want, d, kind):
    need_gpu()
    fgs = lib()
    if want == ("db",) and kind == "rms":
        pytest.skip("an RMS norm has no bias")
    x, _, w, _, dy, _ = _inputs(40, d, "bf16")
    full = _backward(fgs, kind, "bf16", x, None, w, dy, None)
    got = _backward(fgs, kind, "bf16", x, None, w, dy, None, want=want)
    for name in full:
        if got[name] is not None:
            assert torch.equal(got[name], full[name])


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("d", [96, 999, 7168, 20000])
def test_backward_in_place(d, kind):
    """dx may be x, the residual, dy or dh."""
    need_gpu()
    fgs = lib()
    x, r, w, _, dy, dh = _inputs(320, d, "bf16")
    full = _backward(fgs, kind, "bf16", x, r, w, dy, dh)
    for at in range(4):
        t = [v.cuda() for v in (x, r, dy, dh)]
        got = _backward(fgs, kind, "bf16", t[0], t[1], w, t[2], t[3], dx=t[at])
        for name in full:
            assert full[name] is None or torch.equal(got[name], full[name])


ODD = [(3001, 257, "bf16"), (3002, 262, "bf16"), (3007, 1001, "bf16"), (3003, 1002, "bf16"),
       (3005, 1001, "f32"), (3010, 258, "f32"), (3004, 3333, "bf16"), (1603, 7001, "bf16"),
       (1540, 8175, "bf16"), (1540, 8177, "bf16"), (1029, 8183, "f32"), (400, 8003, "f32"),
       (2000, 1001, "bf16"), (20001, 300, "bf16"), (19503, 301, "bf16")]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("residual,dh", [(False, True), (True, False)])
@pytest.mark.parametrize("T,d,dtype", ODD)
def test_backward_many_odd_rows(T, d, dtype, residual, dh, kind):
    """Rows that begin inside a 16-byte chunk, in every place of it; the last row
    ends where the tensors do."""
    need_gpu()
    fgs = lib()
    x, r, w, _, dy, g = _inputs(T, d, dtype)
    r, g = r if residual else None, g if dh else None
    got = _backward(fgs, kind, dtype, x, r, w, dy, g)
    _check_backward(kind, dtype, x, r, w, dy, g, got)
    for at, src in (("dy", dy), ("x", x)):  # dx in place of an input
        t = src.cuda()
        again = _backward(fgs, kind, dtype, t if at == "x" else x, r, w, t if at == "dy" else dy, g,
                          dx=t)
        for name in got:
            assert got[name] is None or torch.equal(got[name], again[name])


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d,dtype", [(3001, 1001, "bf16"), (3006, 1002, "bf16"), (3003, 999, "f32")])
def test_backward_odd_rows_keep_to_themselves(T, d, dtype, kind):
    """A row of infinities and NaN stays in its own dx."""
    need_gpu()
    fgs = lib()
    x, r, w, _, dy, dh = _inputs(T, d, dtype)
    full = _backward(fgs, kind, dtype, x, r, w, dy, dh)["dx"]
    for row in (0, 700, T - 1):
        a = [t.clone() for t in (x, r, dy, dh)]
        for t, v in zip(a, (float("nan"), float("inf"), float("nan"), float("inf"))):
            t[row] = v
        got = _backward(fgs, kind, dtype, a[0], a[1], w, a[2], a[3])["dx"]
        keep = torch.arange(T) != row
        assert torch.equal(got[keep], full[keep])
        assert not got[row].isfinite().any()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d,dtype", [(1030, 1032, "bf16"), (1027, 520, "f32"), (2455, 136, "bf16")])
def test_backward_many_rows_in_place(T, d, dtype, kind):
    """dx in place of each input, and some of the outputs alone, where a block
    keeps copies of its next rows under way."""
    need_gpu()
    fgs = lib()
    x, r, w, _, dy, dh = _inputs(T, d, dtype)
    full = _backward(fgs, kind, dtype, x, r, w, dy, dh)
    for at in range(4):
        t = [v.cuda() for v in (x, r, dy, dh)]
        got = _backward(fgs, kind, dtype, t[0], t[1], w, t[2], t[3], dx=t[at])
        for name in full:
            assert full[name] is None or torch.equal(got[name], full[name])
    for want in (("dw",), ("dw", "db"), ("dx", "dw"), ("dx", "db")):
        if kind == "rms" and "db" in want:
            continue
        got = _backward(fgs, kind, dtype, x, r, w, dy, dh, want=want)
        for name in want:
            assert torch.equal(got[name], full[name])


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d,dtype", [(5, 7168, "f32"), (40, 20000, "bf16"), (1500, 200, "bf16"),
                                       (3000, 256, "f32"), (1030, 1032, "bf16"), (1027, 4096, "f32")])
def test_backward_small_values(T, d, dtype, kind):
    """Rows of 2^-65 with eps 0: the inverse root's square is past fp32's range,
    the gradient is not.

    The squares, above 2^-131 in the mean, are subnormal: each of the d + 64 sums
    is off by half of 2^-149, which is 1.4 2^-150 of the mean for d >= 200, and so
    is the mean's own rounding, 2^-150.  Relative to the variance 2^-17.7, to its
    root 2^-18.7; 2^-18 is allowed."""
    need_gpu()
    fgs = lib()
    x, _, w, _, dy, dh = _inputs(T, d, dtype)
    x = x * 2.0 ** -62  # exact: rows of 2^-65 to 2^-59
    got = _backward(fgs, kind, dtype, x, None, w, dy, dh, eps=0.0)
    X, W, DY, DH = n64(x), n64(w), n64(dy), n64(dh)
    want, lim = norm_backward64(kind, X, None, W, 0.0, DY, DH)
    _, v, r, _ = norm64(kind, X, None, W, None, 0.0)
    g = DY * W
    c = (g * v).mean(1, keepdims=True)
    root = 2.0 ** -18
    more = (root * (r * np.abs(want[0] / r) + 2 * r * np.abs(v * c)) * 1.01,
            root * np.abs(DY * v).sum(0), 0.0)
    for name, a, b, e, rounding in zip(("dx", "dw", "db"), want, lim, more, (U[dtype], u, u)):
        if got[name] is not None:
            close(got[name], a, b + e, rounding)


def test_backward_repeats():
    """The same sums every time, and on a workspace of any contents."""
    need_gpu()
    fgs = lib()
    for T, d in ((2000, 1024), (700, 1024), (3000, 200)):
        x, r, w, _, dy, dh = _inputs(T, d, "bf16")
        a = _backward(fgs, "layer", "bf16", x, r, w, dy, dh)
        for _ in range(5):
            b = _backward(fgs, "layer", "bf16", x, r, w, dy, dh)
            assert all(torch.equal(a[k], b[k]) for k in a)


def test_backward_values():
    """Constant and zero rows; an infinity in one row stays in its dx."""
    need_gpu()
    fgs = lib()
    d = 384
    x, _, w, _, dy, dh = _inputs(8, d, "f32")
    x[0], x[1] = 3.0, 0.0
    dy[2] = 0.0
    for kind in ("rms", "layer"):
        got = _backward(fgs, kind, "f32", x, None, w, dy, dh)
        _check_backward(kind, "f32", x, None, w, dy, dh, got)
        y = dy.clone()
        y[4, 3] = float("inf")
        bad = _backward(fgs, kind, "f32", x, None, w, y, dh, want=("dx",))["dx"]
        assert not bad[4].isfinite().all()
        keep = [0, 1, 2, 3, 5, 6, 7]
        assert torch.equal(bad[keep], got["dx"][keep])


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_backward_by_differences(kind):
    """<dx, V> + <dw, W> + <db, B> against central differences of the norm in
    fp64."""
    need_gpu()
    fgs = lib()
    T, d = 6, 40
    x, _, w, b, dy, _ = _inputs(T, d, "f32")
    got = _backward(fgs, kind, "f32", x, None, w, dy, None)
    rng = np.random.default_rng(4)
    V, W, B = rng.standard_normal((T, d)), rng.standard_normal(d), rng.standard_normal(d)
    if kind == "rms":
        B[:] = 0.0

    def loss(t):
        return (norm64(kind, n64(x) + t * V, None, n64(w) + t * W, n64(b) + t * B, EPS)[3]
                * n64(dy)).sum()

    # fourth-order differences, at two steps: their distance bounds the error left
    def slope(h):
        return (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)

    num, other = slope(1e-3), slope(2e-3)
    dirs = [V, W, B]
    (_, lim) = norm_backward64(kind, n64(x), None, n64(w), EPS, n64(dy), None)
    names = ("dx", "dw", "db")
    val = sum((n64(got[k]) * v).sum() for k, v in zip(names, dirs) if got[k] is not None)
    bound = sum(((e + u * np.abs(n64(got[k]))) * np.abs(v)).sum()
                for k, e, v in zip(names, lim, dirs) if got[k] is not None)
    assert abs(val - num) <= bound + abs(num - other) + 1e-9 * abs(num)


def test_forward_and_backward_captured():
    """Forward and backward captured on one workspace and replayed on new rows,
    while another workspace serves a second stream."""
    need_gpu()
    fgs = lib()
    T, d = 500, 1024
    x, r, w, b, dy, dh = (t.cuda() for t in _inputs(T, d, "bf16"))
    n = fgs.moe_norm_backward_workspace_size(T, d)

    def buffers():
        e = lambda: torch.empty((T, d), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        return dict(h=e(), y=e(), dx=e(), dw=torch.empty(d, device="cuda"),
                    db=torch.empty(d, device="cuda"),
                    ws=torch.zeros(n, dtype=torch.uint8, device="cuda"))

    def step(o, stream=None):
        fgs.moe_add_layernorm(fgs.MOE_BF16, T, d, x, r, w, b, EPS, o["h"], o["y"], stream=stream)
        fgs.moe_norm_backward(1, fgs.MOE_BF16, T, d, o["h"], None, w, EPS, dy, dh, o["dx"],
                              o["dw"], o["db"], o["ws"], n, stream=stream)

    one, two, three = buffers(), buffers(), buffers()
    step(one)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(one)
    for seed in (5, 6):
        for t, v in zip((x, r, dy, dh), [_inputs(T, d, "bf16", seed)[i] for i in (0, 1, 4, 5)]):
            t.copy_(v)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graph.replay()
        step(two, side)  # at the same time, on its own buffers
        torch.cuda.synchronize()
        step(three)
        torch.cuda.synchronize()
        for k in ("h", "y", "dx", "dw", "db"):
            assert torch.equal(one[k], three[k]) and torch.equal(two[k], three[k])


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d", [(3000, 1032), (3001, 1001), (20001, 136)])
def test_many_rows_captured_beside_another_stream(T, d, kind):
    """A captured call replayed on new rows while the same call runs on a second
    stream with its own buffers."""
    need_gpu()
    fgs = lib()
    x, r, w, b, dy, dh = (t.cuda() for t in _inputs(T, d, "bf16"))
    n = fgs.moe_norm_backward_workspace_size(T, d)

    def buffers():
        e = lambda: torch.empty((T, d), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        return dict(y=e(), dx=e(), dw=torch.empty(d, device="cuda"), db=torch.empty(d, device="cuda"),
                    ws=torch.zeros(n, dtype=torch.uint8, device="cuda"))

    def step(o, stream=None):
        fgs.moe_add_layernorm(fgs.MOE_BF16, T, d, x, r, w, b, EPS, None, o["y"], stream=stream)
        fgs.moe_norm_backward(KIND[kind], fgs.MOE_BF16, T, d, x, r, w, EPS, dy, dh, o["dx"], o["dw"],
                              o["db"] if kind == "layer" else None, o["ws"], n, stream=stream)

    one, two, three = buffers(), buffers(), buffers()
    step(one)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(one)
    for t, v in zip((x, r, dy, dh), [_inputs(T, d, "bf16", 5)[i] for i in (0, 1, 4, 5)]):
        t.copy_(v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        graph.replay()
        step(two, side)
    torch.cuda.synchronize()
    step(three)
    torch.cuda.synchronize()
    for k in ("y", "dx", "dw") + (("db",) if kind == "layer" else ()):
        assert torch.equal(one[k], three[k]) and torch.equal(two[k], three[k])
    assert fgs.moe_get_device_status(one["ws"]) == 0


def test_long_rows_offsets():
    """Elements past 2^31: rows x columns beyond 32 bits."""
    need_gpu()
    fgs = lib()
    T, d = 300_001, 7168  # 2.15e9 elements
    dt = torch.bfloat16
    x = torch.zeros((T, d), dtype=dt, device="cuda")
    dy = torch.zeros((T, d), dtype=dt, device="cuda")
    gen = torch.Generator().manual_seed(2)
    last = torch.randn((3, d), generator=gen).to(dt)
    g = torch.randn((3, d), generator=gen).to(dt)
    x[-3:], dy[-3:] = last.cuda(), g.cuda()
    w, b = torch.ones(d, dtype=dt), torch.zeros(d, dtype=dt)
    y = torch.empty_like(x)
    fgs.moe_add_layernorm(fgs.MOE_BF16, T, d, x, None, w.cuda(), b.cuda(), EPS, None, y)
    _check_forward("bf16", last, None, w, b, None, y[-3:].cpu())
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    n = fgs.moe_norm_backward_workspace_size(T, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    fgs.moe_norm_backward(1, fgs.MOE_BF16, T, d, x, None, w.cuda(), EPS, dy, None, y, dw, db, ws, n)
    # rows of zeros add nothing to the sums, whatever their chain
    _check_backward("layer", "bf16", last, None, w, g, None,
                    {"dx": y[-3:].cpu(), "dw": dw.cpu(), "db": db.cpu()})
