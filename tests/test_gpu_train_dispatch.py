"""The rows in expert order, and the way back through the combine and the gate
weights, against plain fp64 forms."""
import numpy as np
import pytest
import torch

from _gpu_common import lib, need_gpu, workspace
from _train_common import DT, U, chain, close, n64, router_backward64, routing, slots, u

pytestmark = pytest.mark.gpu

SCALE = 2.827


def _cfg(fgs, d, K, E, dtype, **kw):
    base = dict(d_model=d, d_ff=64, E_routed=E, K=K,
                dtype=fgs.MOE_BF16 if dtype == "bf16" else fgs.MOE_F32)
    base.update(kw)
    return fgs.config(**base)


SHAPES = [  # T, K, E, D, dtype, share of rejected pairs
    (1, 1, 1, 128, "bf16", 0.0),
    (1, 8, 384, 7168, "bf16", 0.0),
    (1, 1, 4, 32, "f32", 0.0),
    (3, 2, 5, 96, "f32", 0.4),
    (7, 16, 63, 3584, "bf16", 0.1),
    (65, 32, 64, 256, "bf16", 0.05),
    (301, 6, 64, 1920, "f32", 0.02),
    (1025, 9, 16, 384, "bf16", 0.0),
    (1500, 3, 7, 1152, "f32", 0.0),
]


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("T,K,E,D,dtype,bad", SHAPES)
def test_gather(T, K, E, D, dtype, bad, weights):
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(T + K + D)
    inv, kept = slots(routing(T, K, E, gen, bad), E)
    x = torch.randn((T, D), generator=gen).to(DT[dtype])
    x.view(-1)[:3] = torch.tensor([float("nan"), float("inf"), -0.0])
    w = torch.randn((T, K), generator=gen)
    xp = torch.full((T * K + 1, D), 7.0, dtype=DT[dtype], device="cuda")
    wp = torch.full((T * K + 1,), 7.0, device="cuda")
    fgs.moe_gather(_cfg(fgs, D, K, E, dtype), T, x.cuda(), torch.from_numpy(inv).cuda(),
                   w.cuda() if weights else None, xp, wp if weights else None)
    pairs = np.flatnonzero(inv >= 0)
    want = torch.full((T * K + 1, D), 7.0, dtype=DT[dtype])
    want[inv[pairs]] = x[pairs // K]
    wants = torch.full((T * K + 1,), 7.0)
    if weights:
        wants[inv[pairs]] = w.view(-1)[pairs]
    as_bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(xp.cpu().view(as_bits), want.view(as_bits))  # rows behind the last included
    assert torch.equal(wp.cpu(), wants)


def test_gather_ignores_slots_outside():
    """Slots outside [0, T K) write nothing, whatever their size."""
    need_gpu()
    fgs = lib()
    T, K, D = 4, 2, 128
    inv = torch.tensor([0, -1, T * K, 2 ** 31 - 1, -2 ** 31, 5, 7, 3], dtype=torch.int32)
    x = torch.randn((T, D)).bfloat16()
    xp = torch.zeros((T * K, D), dtype=torch.bfloat16, device="cuda")
    fgs.moe_gather(_cfg(fgs, D, K, 4, "bf16"), T, x.cuda(), inv.cuda(), None, xp, None)
    want = torch.zeros((T * K, D), dtype=torch.bfloat16)
    want[0], want[5], want[7], want[3] = x[0], x[2], x[3], x[3]
    assert torch.equal(xp.cpu(), want)


@pytest.mark.parametrize("T,K,E,D,dtype,bad", SHAPES)
def test_gather_gradient_is_the_combine(T, K, E, D, dtype, bad):
    """dx[t] = sum_k dx_perm[inv], with the shared experts' gradients added."""
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(T + K + D)
    inv, _ = slots(routing(T, K, E, gen, bad), E)
    g = torch.randn((T * K, D), generator=gen).to(DT[dtype])
    sh = torch.randn((1, T, D), generator=gen).to(DT[dtype])
    dx = torch.empty((T, D), dtype=DT[dtype], device="cuda")
    fgs.moe_combine(_cfg(fgs, D, K, E, dtype, E_shared=1, d_ff_shared=64), T, g.cuda(),
                    torch.from_numpy(inv).cuda(), None, sh.cuda(), dx)
    rows = np.where(inv[:, None] >= 0, n64(g)[np.maximum(inv, 0)], 0.0).reshape(T, K, D)
    want = rows.sum(1) + n64(sh)[0]
    close(dx, want, (K + 1) * u * (np.abs(rows).sum(1) + np.abs(n64(sh)[0])), U[dtype])


def _combine_backward(fgs, T, K, E, D, dtype, bad, weights=True, dY=True, dw=True, seed=0):
    gen = torch.Generator().manual_seed(seed + T + K + D)
    inv, kept = slots(routing(T, K, E, gen, bad), E)
    dy = torch.randn((T, D), generator=gen).to(DT[dtype])
    Y = (torch.randn((T * K, D), generator=gen) * 3).to(DT[dtype])
    w = torch.randn((T, K), generator=gen) if weights else None
    out = torch.full((T * K + 1, D), 7.0, dtype=DT[dtype], device="cuda") if dY else None
    dwo = torch.full((T * K + 1,), 7.0, device="cuda") if dw else None
    fgs.moe_combine_backward(_cfg(fgs, D, K, E, dtype), T, dy.cuda(), Y.cuda() if dw else None,
                             torch.from_numpy(inv).cuda(), None if w is None else w.cuda(), out, dwo)
    return inv, dy, Y, w, out, dwo


@pytest.mark.parametrize("weights,dY,dw", [(True, True, True), (False, True, True),
                                           (True, False, True), (True, True, False)])
@pytest.mark.parametrize("T,K,E,D,dtype,bad", SHAPES)
def test_combine_backward(T, K, E, D, dtype, bad, weights, dY, dw):
    need_gpu()
    fgs = lib()
    inv, dy, Y, w, out, dwo = _combine_backward(fgs, T, K, E, D, dtype, bad, weights, dY, dw)
    pairs = np.flatnonzero(inv >= 0)
    g, y = n64(dy)[pairs // K], n64(Y)[inv[pairs]]
    if dY:
        want = np.full((T * K + 1, D), 7.0)
        want[inv[pairs]] = g * (n64(w).reshape(-1)[pairs][:, None] if weights else 1.0)
        # the product in fp32, then the output's rounding
        close(out, want, u * np.abs(want), U[dtype])
    if dw:
        want, lim = np.zeros(T * K + 1), np.zeros(T * K + 1)
        want[-1] = 7.0
        want[pairs] = (g * y).sum(1)
        lim[pairs] = (chain(D) + 1) * u * np.abs(g * y).sum(1)
        close(dwo, want, lim, 0.0)


def test_combine_backward_in_place():
    """dY may be Y."""
    need_gpu()
    fgs = lib()
    for T, K, E, D, dtype, bad in SHAPES[4:7]:
        inv, dy, Y, w, out, dwo = _combine_backward(fgs, T, K, E, D, dtype, bad)
        Yd = torch.cat((Y, Y[:1])).cuda()
        dw2 = torch.full_like(dwo, 7.0)
        fgs.moe_combine_backward(_cfg(fgs, D, K, E, dtype), T, dy.cuda(), Yd,
                                 torch.from_numpy(inv).cuda(), w.cuda(), Yd, dw2)
        kept = torch.from_numpy(np.sort(inv[inv >= 0])).long()
        assert torch.equal(Yd.cpu()[kept], out.cpu()[kept]) and torch.equal(dw2, dwo)


def test_combine_backward_by_differences():
    """<dL/dY, V> + <dL/dw, W> against central differences of the combine, in
    fp64 (L is bilinear in Y and w, so the difference is exact but for its
    rounding)."""
    need_gpu()
    fgs = lib()
    T, K, E, D = 20, 4, 9, 160
    inv, dy, Y, w, out, dwo = _combine_backward(fgs, T, K, E, D, "f32", 0.1)
    rng = np.random.default_rng(1)
    V, W = rng.standard_normal((T * K, D)), rng.standard_normal((T, K))

    def loss(y, wt):
        rows = np.where(inv[:, None] >= 0, y[np.maximum(inv, 0)], 0.0).reshape(T, K, D)
        return ((rows * wt[:, :, None]).sum(1) * n64(dy)).sum()

    h = 1e-3
    num = (loss(n64(Y) + h * V, n64(w) + h * W) - loss(n64(Y) - h * V, n64(w) - h * W)) / (2 * h)
    kept = inv[inv >= 0]
    a = (n64(out)[kept] * V[kept]).sum()
    b = (n64(dwo)[:-1] * W.reshape(-1)).sum()
    # dY is within its two roundings, dw within its sum's chain
    lim = 2 * u * np.abs(n64(out)[kept] * V[kept]).sum()
    products = np.abs(n64(Y)[kept] * np.repeat(n64(dy), K, 0)[inv >= 0]).sum(1)
    lim += (chain(D) + 1) * u * (products * np.abs(W.reshape(-1))[inv >= 0]).sum()
    assert abs(a + b - num) <= lim + 1e-9 * abs(num)


def test_combine_backward_values_that_are_not_finite():
    """An infinity or NaN stays in its token's pairs."""
    need_gpu()
    fgs = lib()
    T, K, D = 5, 2, 256
    inv = torch.arange(T * K, dtype=torch.int32)
    dy, Y = torch.ones((T, D)).bfloat16(), torch.ones((T * K, D)).bfloat16()
    dy[1, 7] = float("inf")
    Y[4, 9] = float("nan")  # token 2, pair 0
    out = torch.empty((T * K, D), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((T, K), device="cuda")
    fgs.moe_combine_backward(_cfg(fgs, D, K, 4, "bf16"), T, dy.cuda(), Y.cuda(), inv.cuda(),
                             torch.full((T, K), 2.0, device="cuda"), out, dw)
    want = torch.full((T, K), float(D))
    want[1] = float("inf")
    want[2, 0] = float("nan")
    torch.testing.assert_close(dw.cpu(), want, rtol=0, atol=0, equal_nan=True)
    rows = torch.full((T * K, D), 2.0)
    rows[2:4, 7] = float("inf")
    assert torch.equal(out.float().cpu(), rows)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,K,E,bad", [(1, 1, 1, 0.0), (1, 8, 384, 0.0), (3, 2, 5, 0.3),
                                       (129, 32, 33, 0.1), (1000, 16, 896, 0.0), (77, 6, 63, 0.0),
                                       (50, 4, 1024, 1.0)])
def test_router_backward(T, K, E, bad, renorm):
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(T + K + E)
    idx = routing(T, K, E, gen, bad)
    z = torch.randn((T, E), generator=gen) * 3
    dw = torch.randn((T, K), generator=gen)
    dz = torch.full((T + 1, E), 7.0, device="cuda")
    cfg = _cfg(fgs, 128, K, E, "bf16", norm_topk_prob=renorm)
    fgs.moe_router_backward(cfg, T, z.cuda(), idx.cuda(), dw.cuda(), dz)
    want, bound = router_backward64(n64(z), idx.numpy(), n64(dw), E, SCALE, renorm and K > 1)
    assert (dz[T] == 7.0).all()
    close(dz[:T], want, bound, u)
    assert (dz[:T].cpu().numpy()[want == 0] == 0).all()


def test_router_backward_far_logits():
    """Logits whose sigmoids, or their rests, vanish or saturate."""
    need_gpu()
    fgs = lib()
    z = torch.tensor([[-200.0, -100.0, -60.0, -30.0], [200.0, 100.0, 60.0, 30.0],
                      [-200.0, 200.0, 0.0, -50.0], [-45.0, -46.0, -47.0, -48.0],
                      [float("-inf"), 3.0, float("inf"), 0.0]])
    T, E = z.shape
    idx = torch.arange(E, dtype=torch.int32).repeat(T, 1)
    dw = torch.tensor([[1.0, -2.0, 3.0, -4.0]]).repeat(T, 1)
    dz = torch.empty((T, E), device="cuda")
    fgs.moe_router_backward(_cfg(fgs, 128, E, E, "bf16"), T, z.cuda(), idx.cuda(), dw.cuda(), dz)
    want, bound = router_backward64(n64(z), idx.numpy(), n64(dw), E, SCALE, True)
    close(dz, want, bound, u)


def test_router_backward_repeated_expert():
    """An expert listed twice receives the sum of its pairs' gradients."""
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(3)
    idx = torch.tensor([[2, 2, 0, 2], [1, 9, 1, -1], [3, 3, 3, 3]], dtype=torch.int32)
    z, dw = torch.randn((3, 4), generator=gen), torch.randn((3, 4), generator=gen)
    dz = torch.empty((3, 4), device="cuda")
    fgs.moe_router_backward(_cfg(fgs, 128, 4, 4, "bf16"), 3, z.cuda(), idx.cuda(), dw.cuda(), dz)
    want, bound = router_backward64(n64(z), idx.numpy(), n64(dw), 4, SCALE, True)
    close(dz, want, bound * 4, 4 * u)


def test_router_backward_by_differences():
    need_gpu()
    fgs = lib()
    T, K, E = 12, 5, 24
    gen = torch.Generator().manual_seed(5)
    idx = routing(T, K, E, gen)
    z, dw = torch.randn((T, E), generator=gen), torch.randn((T, K), generator=gen)
    dz = torch.empty((T, E), device="cuda")
    fgs.moe_router_backward(_cfg(fgs, 128, K, E, "bf16"), T, z.cuda(), idx.cuda(), dw.cuda(), dz)
    v = np.random.default_rng(2).standard_normal((T, E))

    def loss(zz):
        s = 1 / (1 + np.exp(-np.take_along_axis(zz, idx.numpy().astype(np.int64), 1)))
        return (SCALE * s / (s.sum(1, keepdims=True) + 1e-20) * n64(dw)).sum()

    h = 1e-4
    num = (loss(n64(z) + h * v) - loss(n64(z) - h * v)) / (2 * h)
    _, bound = router_backward64(n64(z), idx.numpy(), n64(dw), E, SCALE, True)
    # the difference's own error is h^2 / 6 of a third derivative that is at
    # most a few |dw| |v|^3 a pair
    lim = (bound * np.abs(v)).sum() + h * h * SCALE * np.abs(n64(dw)).sum() * (np.abs(v) ** 3).max()
    assert abs((n64(dz) * v).sum() - num) <= lim


def test_gate_weights_of_the_router():
    """The weights whose gradient router_backward takes are the router's own."""
    need_gpu()
    fgs = lib()
    T, K, E = 40, 4, 32
    gen = torch.Generator().manual_seed(8)
    z = torch.randn((T, E), generator=gen).cuda()
    idx = torch.empty((T, K), dtype=torch.int32, device="cuda")
    w = torch.empty((T, K), device="cuda")
    cfg = _cfg(fgs, 128, K, E, "bf16")
    fgs.moe_router_from_logits(cfg, T, z, torch.zeros(E, device="cuda"), idx, w)
    z64 = z.double().cpu().requires_grad_()
    s = torch.sigmoid(z64.gather(1, idx.cpu().long()))
    w64 = SCALE * s / (s.sum(1, keepdim=True) + 1e-20)
    assert (w64.detach() - w.cpu().double()).abs().max() <= 1e-6
    dw = torch.randn((T, K), generator=gen)
    (w64 * dw.double()).sum().backward()
    dz = torch.empty((T, E), device="cuda")
    fgs.moe_router_backward(cfg, T, z, idx, dw.cuda(), dz)
    _, bound = router_backward64(n64(z), idx.cpu().numpy(), n64(dw), E, SCALE, True)
    close(dz, z64.grad.numpy(), bound, u)


def test_captured_and_on_another_stream():
    """Permute, gather and the combine's gradient on a side stream, captured
    and replayed on new contents of the same buffers."""
    need_gpu()
    fgs = lib()
    T, K, E, D = 100, 4, 16, 512
    cfg = _cfg(fgs, D, K, E, "bf16")
    ws, nws = workspace(cfg, T)
    gen = torch.Generator().manual_seed(11)
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    perm, inv = torch.empty(T * K, **i32), torch.empty(T * K, **i32)
    idx = routing(T, K, E, gen).cuda()
    x = torch.randn((T, D), generator=gen).bfloat16().cuda()
    w = torch.randn((T, K), generator=gen).cuda()
    xp, dY = (torch.zeros((T * K, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wp, dw = torch.zeros(T * K, device="cuda"), torch.zeros((T, K), device="cuda")

    def step():
        fgs.moe_permute(cfg, T, idx, counts, offsets, perm, inv, ws, nws)
        fgs.moe_gather(cfg, T, x, inv, w, xp, wp)
        fgs.moe_combine_backward(cfg, T, x, xp, inv, w, dY, dw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        gen.manual_seed(seed)
        idx.copy_(routing(T, K, E, gen))
        x.copy_(torch.randn((T, D), generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        ref, _ = slots(idx.cpu(), E)
        assert np.array_equal(inv.cpu().numpy(), ref)
        want = torch.empty((T * K, D), dtype=torch.bfloat16)
        want[ref.astype(np.int64)] = x.cpu().repeat_interleave(K, 0)
        assert torch.equal(xp.cpu(), want)
        x64 = n64(x)
        close(dw, np.repeat((x64 * x64).sum(1, keepdims=True), K, 1),
              (chain(D) + 1) * u * (x64 * x64).sum(1, keepdims=True), 0.0)


def test_offsets_past_32_bits():
    """Rows in expert order of more than 2^32 elements: the gather and the
    combine's gradient, checked at the first and last pairs of every expert."""
    need_gpu()
    fgs = lib()
    T, K, E, D = 40000, 16, 32, 7168  # 4.59e9 elements
    cfg = _cfg(fgs, D, K, E, "bf16")
    gen = torch.Generator().manual_seed(3)
    idx = routing(T, K, E, gen)
    inv_host, kept = slots(idx, E)
    assert kept * D > 2 ** 32
    inv = torch.from_numpy(inv_host).cuda()
    x = torch.randn((T, D), device="cuda", dtype=torch.bfloat16)
    w = torch.rand((T, K), device="cuda")
    xp = torch.empty((kept, D), dtype=torch.bfloat16, device="cuda")
    wp = torch.empty(kept, device="cuda")
    fgs.moe_gather(cfg, T, x, inv, w, xp, wp)
    pairs = torch.cat([torch.arange(64), torch.arange(T * K - 64, T * K)]).cuda()
    at = inv.long()
    pairs = torch.cat([pairs, at.argsort()[torch.arange(0, kept, 4999, device="cuda")],
                       at.argsort()[-64:]])
    rows = at[pairs]
    assert torch.equal(xp[rows], x[pairs // K])
    assert torch.equal(wp[rows], w.reshape(-1)[pairs])
    dy = torch.randn((T, D), device="cuda", dtype=torch.bfloat16)
    dw = torch.empty((T, K), device="cuda")
    Y = xp[rows].clone()
    fgs.moe_combine_backward(cfg, T, dy, xp, inv, w, xp, dw)  # dY in place of Y
    g = dy[pairs // K].double()
    close(xp[rows].cpu(), n64(w.reshape(-1)[pairs, None].double() * g),
          0.0, U["bf16"] + 2 * u)  # the product in fp32, then rounded
    want = (Y.double() * g)
    close(dw.reshape(-1)[pairs].cpu(), n64(want.sum(1)),
          n64(want.abs().sum(1)) * (chain(D) + 2) * u, u)


def test_router_backward_offsets_past_32_bits():
    need_gpu()
    fgs = lib()
    T, K, E = 4_800_001, 8, 896  # 4.3e9 logits
    z = torch.zeros((T, E), device="cuda")
    gen = torch.Generator().manual_seed(4)
    n = 50
    tail = torch.randn((n, E), generator=gen)
    idx = routing(n, K, E, gen)
    g = torch.randn((n, K), generator=gen)
    z[-n:] = tail.cuda()
    all_idx = torch.zeros((T, K), dtype=torch.int32, device="cuda")
    all_idx[-n:] = idx.cuda()
    dw = torch.zeros((T, K), device="cuda")
    dw[-n:] = g.cuda()
    dz = torch.full((T, E), 9.0, device="cuda")
    cfg = _cfg(fgs, 128, K, E, "bf16")
    fgs.moe_router_backward(cfg, T, z, all_idx, dw, dz)
    want, lim = router_backward64(n64(tail), idx.numpy(), n64(g), E,
                                  cfg.routed_scaling_factor, True)
    close(dz[-n:].cpu(), want, lim, u)
    assert int((dz[:-n] != 0).sum()) == 0
