"""Plain fp64 forms of the training operators and the error bounds their tests
use (not collected as a test module).  u = 2^-24 is half a step of fp32: the
most by which one rounded operation is off, relative to its result."""
import numpy as np
import torch

from _int4_common import U_BF16, U_F32, close  # noqa: F401

u = U_F32
U = {"bf16": U_BF16, "f32": U_F32}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def n64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def routing(T, K, E, gen, bad=0.0):
    """[T, K] distinct experts a token, some indices outside [0, E)."""
    idx = torch.rand((T, E), generator=gen).topk(K, dim=1).indices.to(torch.int32)
    if bad:
        wrong = torch.rand((T, K), generator=gen) < bad
        idx[wrong] = torch.where(torch.rand((int(wrong.sum()),), generator=gen) < 0.5, E, -3).int()
    return idx


def slots(idx, E):
    """(inv, kept) of the stable sort of the pairs by expert; inv -1 for a pair
    outside [0, E)."""
    flat = idx.reshape(-1).numpy()
    ok = (flat >= 0) & (flat < E)
    order = np.flatnonzero(ok)[np.argsort(flat[ok], kind="stable")]
    inv = np.full(flat.size, -1, np.int32)
    inv[order] = np.arange(order.size, dtype=np.int32)
    return inv, order.size


def chain(n):
    """Roundings a term of a sum over n passes through at most: the sums are
    split over a warp's lanes at least, each part added in its order, then in
    a tree or over a block's 32 warps."""
    return n / 32 + 32


def norm64(kind, x, residual, w, b, eps):
    """(s, u, r, y) of the norm of fp64 rows."""
    s = x + (residual if residual is not None else 0.0)
    c = s - s.mean(1, keepdims=True) if kind == "layer" else s
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
        y = c * r * w + (b if b is not None else 0.0)
        return s, c * r, r, y


def norm_errors(kind, s, r, d, eps):
    """Bounds of the fp32 errors: of (s - mu) r elementwise, and of r relative.
    s is one rounded sum; mu a sum of d of them over d; the squares' mean has
    their errors and its chain's; rsqrt is within 2 ulp (4 u)."""
    n = chain(d)
    es = u * np.abs(s)
    if kind == "layer":
        mu = s.mean(1, keepdims=True)
        em = (n + 2) * u * np.abs(s).mean(1, keepdims=True)
        c = s - mu
        es = es + em + u * np.abs(c)
    else:
        c = s
    var = (c * c).mean(1, keepdims=True)
    ev = (n + 3) * u * var + 2 * (np.abs(c) * es).mean(1, keepdims=True)
    ev = ev + (es * es).mean(1, keepdims=True) + u * (var + eps)
    rel = 0.5 * ev / np.maximum(var + eps, 1e-300) * 1.01 + 4 * u
    return es * r + np.abs(c) * r * (rel + 2 * u), rel


def norm_backward64(kind, x, residual, w, eps, dy, dh):
    """((dx, dw, db), their bounds) of the norm's gradient."""
    s, v, r, _ = norm64(kind, x, residual, w, None, eps)
    d = x.shape[1]
    ev, rel = norm_errors(kind, s, r, d, eps)
    n = chain(d)
    g = dy * w
    eg = u * np.abs(g)
    mg = g.mean(1, keepdims=True) if kind == "layer" else np.zeros_like(r)
    emg = (n + 2) * u * np.abs(g).mean(1, keepdims=True) if kind == "layer" else 0.0
    c = (g * v).mean(1, keepdims=True)
    ec = (n + 6) * u * np.abs(g * v).mean(1, keepdims=True) + (np.abs(g) * ev).mean(1, keepdims=True)
    ec = ec + (rel + 2 * u) * np.abs(c)
    t = g - mg - v * c
    et = eg + emg + ev * np.abs(c) + np.abs(v) * ec + ev * ec
    et = et + 4 * u * (np.abs(g) + np.abs(mg) + np.abs(v * c))
    dx = r * t + (dh if dh is not None else 0.0)
    edx = r * et * 1.001 + (rel + 3 * u) * np.abs(r * t) + u * np.abs(dx)
    m = chain(x.shape[0])
    dw = (dy * v).sum(0)
    edw = (np.abs(dy) * ev).sum(0) + (m + 2) * u * (np.abs(dy * v)).sum(0)
    db = dy.sum(0)
    edb = (m + 1) * u * np.abs(dy).sum(0)
    return (dx, dw, db), (edx, edw, edb)


def router_backward64(z, idx, dw, E, scale, renorm):
    """(dz, bound): the gradient of the gate weights to the logits.  In fp32 an
    exponential is within 2 ulp, 4 u, its square within 9 u, and a sigmoid or
    its rest, e / (1 + e) or 1 / (1 + e), within 16 u; their sum within 21, p
    within 38, mean within 44 of sum p |dw|, and the product of p, the
    difference and the rest within 38 + 16 + 4 more: 128 u of the sizes
    together."""
    T, K = idx.shape
    dz, bound = np.zeros((T, E)), np.zeros((T, E))
    ok = (idx >= 0) & (idx < E)
    at = np.where(ok, idx, 0)
    zk = np.take_along_axis(z, at, 1)
    with np.errstate(over="ignore"):
        s, rest = 1 / (1 + np.exp(-zk)), 1 / (1 + np.exp(zk))
    p = np.where(ok, s, 0.0)
    d = np.where(ok, dw, 0.0)
    mean = np.zeros((T, 1))
    size = np.abs(d)
    if renorm:
        p = p / (p.sum(1, keepdims=True) + 1e-20)
        mean = (p * d).sum(1, keepdims=True)
        size = size + (p * np.abs(d)).sum(1, keepdims=True)
    g = scale * p * (d - mean) * rest
    e = 128 * u * scale * p * size * rest + 1e-37
    for k in range(K):
        t = np.flatnonzero(ok[:, k])
        dz[t, idx[t, k]] += g[t, k]
        bound[t, idx[t, k]] += e[t, k]
    return dz, bound
