"""The training operators together: a step of a small layer whose expert
products are the caller's, from the norm through the router, the sort, the
experts, the combine and back, and the AdamW update, against fp64 autograd."""
import pytest
import torch

from _gpu_common import lib, need_gpu, workspace
from _train_common import U_BF16

pytestmark = pytest.mark.gpu

EPS = 1e-6
SCALE = 2.827


def _setup(T, d, F, E, K, gen):
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    p = {"norm": 1 + 0.1 * r(d), "bias": 0.1 * r(d), "router": r(E, d) / d ** 0.5,
         "up": r(E, F, d) / d ** 0.5, "down": r(E, d, F) / F ** 0.5, "shared": r(d, d) / d ** 0.5}
    return p, r(T, d), r(T, d), r(T, d)


def _forward64(kind, p, a, res, idx, K):
    """(y, h) of the layer in fp64, given the routing."""
    h = a + res
    c = h - h.mean(1, keepdim=True) if kind == "layer" else h
    x = c / torch.sqrt((c * c).mean(1, keepdim=True) + EPS) * p["norm"]
    if kind == "layer":
        x = x + p["bias"]
    s = torch.sigmoid((x @ p["router"].t()).gather(1, idx))
    w = SCALE * s / (s.sum(1, keepdim=True) + 1e-20)
    y = x @ p["shared"].t()
    for k in range(K):
        u = torch.einsum("tfd,td->tf", p["up"][idx[:, k]], x)
        u = torch.nn.functional.silu(u)
        y = y + w[:, k, None] * torch.einsum("tdf,tf->td", p["down"][idx[:, k]], u)
    return y + h, h


def _step(fgs, kind, p, a, res, g, E, K):
    """One forward and backward pass by the library's calls, the experts'
    products in torch (fp32)."""
    T, d = a.shape
    cfg = fgs.config(d_model=d, d_ff=64, E_routed=E, K=K, E_shared=1, d_ff_shared=64,
                     dtype=fgs.MOE_F32)
    ws, nws = workspace(cfg, T)
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    h, x = e(T, d), e(T, d)
    if kind == "rms":
        fgs.moe_add_rmsnorm(fgs.MOE_F32, T, d, a, res, p["norm"], EPS, h, x)
    else:
        fgs.moe_add_layernorm(fgs.MOE_F32, T, d, a, res, p["norm"], p["bias"], EPS, h, x)
    z = x @ p["router"].t()
    idx, w = torch.empty((T, K), dtype=torch.int32, device="cuda"), e(T, K)
    fgs.moe_router_from_logits(cfg, T, z, torch.zeros(E, device="cuda"), idx, w)
    counts, offsets, perm, inv = i32(E), i32(E + 1), i32(T * K), i32(T * K)
    fgs.moe_permute(cfg, T, idx, counts, offsets, perm, inv, ws, nws)
    xp, Y, y = e(T * K, d), e(T * K, d), e(T, d)
    fgs.moe_gather(cfg, T, x, inv, None, xp)
    off, kept = offsets.tolist(), {}
    for n in range(E):
        rows = xp[off[n]:off[n + 1]]
        u = rows @ p["up"][n].t()
        sig = torch.sigmoid(u)
        kept[n] = (rows, u, sig)
        Y[off[n]:off[n + 1]] = (u * sig) @ p["down"][n].t()
    shared = (x @ p["shared"].t()).unsqueeze(0).contiguous()
    fgs.moe_combine(cfg, T, Y, inv, w, shared, y)
    y += h
    # and back, from g, the gradient of y
    grad = {k: torch.zeros_like(v) for k, v in p.items()}
    dY, dw, dxp, dx, dz = e(T * K, d), e(T, K), e(T * K, d), e(T, d), e(T, E)
    fgs.moe_combine_backward(cfg, T, g, Y, inv, w, dY, dw)
    for n in range(E):
        rows, u, sig = kept[n]
        dy = dY[off[n]:off[n + 1]]
        grad["down"][n] = dy.t() @ (u * sig)
        du = (dy @ p["down"][n]) * sig * (1 + u * (1 - sig))
        grad["up"][n] = du.t() @ rows
        dxp[off[n]:off[n + 1]] = du @ p["up"][n]
    fgs.moe_router_backward(cfg, T, z, idx, dw, dz)
    grad["router"] = dz.t() @ x
    grad["shared"] = g.t() @ x
    extra = (g @ p["shared"] + dz @ p["router"]).unsqueeze(0).contiguous()
    fgs.moe_combine(cfg, T, dxp, inv, None, extra, dx)  # the gradient of the gather
    da = e(T, d)
    nb = fgs.moe_norm_backward_workspace_size(T, d)
    nws2 = torch.empty(nb, dtype=torch.uint8, device="cuda")
    code = fgs.MOE_NORM_RMS if kind == "rms" else fgs.MOE_NORM_LAYER
    fgs.moe_norm_backward(code, fgs.MOE_F32, T, d, h, None, p["norm"], EPS, dx, g, da,
                          grad["norm"], grad["bias"] if kind == "layer" else None, nws2, nb)
    assert fgs.moe_get_device_status(ws) == 0
    return y, idx, da, grad


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d,F,E,K", [(50, 96, 64, 8, 2), (300, 256, 128, 16, 4), (1, 64, 32, 4, 4)])
def test_step(T, d, F, E, K, kind):
    need_gpu()
    fgs = lib()
    gen = torch.Generator().manual_seed(T + d)
    p, a, res, g = _setup(T, d, F, E, K, gen)
    gpu = {k: v.cuda() for k, v in p.items()}
    y, idx, da, grad = _step(fgs, kind, gpu, a.cuda(), res.cuda(), g.cuda(), E, K)
    p64 = {k: v.double().requires_grad_() for k, v in p.items()}
    a64 = a.double().requires_grad_()
    want, _ = _forward64(kind, p64, a64, res.double(), idx.cpu().long(), K)
    (want * g.double()).sum().backward()

    # a dozen fp32 products of up to max(d, F, T K) terms stand between the
    # inputs and any of these; each is off by at most its length's root, taken
    # twelvefold, of 2^-24 of its size, and in the 2-norm they add up
    tol = 12 * 12 * max(d, F, T * K) ** 0.5 * 2.0 ** -24
    def near(got, ref, name):  # noqa: E306
        ref = ref.detach()
        err = (got.cpu().double() - ref).norm() / ref.norm().clamp_min(1e-30)
        assert err <= tol, (name, float(err), tol)

    near(y, want, "y")
    near(da, a64.grad, "da")
    for k, v in p64.items():
        if k != "bias" or kind == "layer":
            near(grad[k], v.grad, k)


@pytest.mark.parametrize("bits", [8, 32])
def test_update_of_all_weights(bits):
    """The gradients of a step into AdamW: fp32 norm and router weights in one
    call, bf16 banks with master copies in another; the first step moves every
    weight by lr in the direction of its gradient."""
    need_gpu()
    fgs = lib()
    T, d, F, E, K = 64, 128, 64, 8, 2
    gen = torch.Generator().manual_seed(3)
    p, a, res, g = _setup(T, d, F, E, K, gen)
    gpu = {k: v.cuda() for k, v in p.items()}
    _, _, _, grad = _step(fgs, "layer", gpu, a.cuda(), res.cuda(), g.cuda(), E, K)
    lr, wd = 1e-3, 0.1

    def states(n):
        if bits == 32:
            return {"exp_avg": torch.zeros(n, device="cuda"),
                    "exp_avg_sq": torch.zeros(n, device="cuda")}
        z = lambda dt, m: torch.zeros(m, dtype=dt, device="cuda")  # noqa: E731
        nb = -(-n // 128)
        return {"exp_avg": z(torch.uint8, n), "exp_avg_sq": z(torch.uint8, n),
                "exp_avg_scale": z(torch.float32, nb), "exp_avg_sq_scale": z(torch.float32, nb)}

    small, banks, before = [], [], {}
    for k, v in gpu.items():
        before[k] = v.double().cpu()
        if v.dim() == 3:
            banks.append({"param": v.bfloat16(), "master": v.clone(), "grad": grad[k],
                          "weight_decay": wd, **states(v.numel())})
        else:
            small.append({"param": v, "grad": grad[k], **states(v.numel())})
    fgs.moe_adamw(fgs.adamw_table(small), fgs.MOE_F32, fgs.MOE_F32, bits, lr, 0.9, 0.99, 1e-12, 1,
                  seed=1)
    fgs.moe_adamw(fgs.adamw_table(banks), fgs.MOE_BF16, fgs.MOE_F32, bits, lr, 0.9, 0.99, 1e-12, 1,
                  seed=1)
    for (k, v), t in zip(gpu.items(), _in_order(gpu, small, banks)):
        decay = 1 - lr * t.get("weight_decay", 0.0)
        gr = grad[k].double().cpu()
        # m / sqrt(v) is the gradient's sign but for eps and a dozen roundings;
        # the factor 1 - lr wd, its product with p and the difference are three more
        want = before[k] * decay - lr * gr / (gr.abs() + 1e-12)
        got = (t["master"] if "master" in t else t["param"]).double().cpu().view(want.shape)
        lim = 2.0 ** -24 * (3 * want.abs() + 15 * lr)
        assert ((got - want).abs() <= lim).all(), k
        if "master" in t:
            low = t["param"].double().cpu()
            assert ((low - got).abs() <= U_BF16 * got.abs() * (1 + 1e-6)).all()


def _in_order(gpu, small, banks):
    small, banks = iter(small), iter(banks)
    return [next(banks) if v.dim() == 3 else next(small) for v in gpu.values()]
