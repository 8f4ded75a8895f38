"""Plain fp64 forms of the 4-bit products and the RMS norm, and the error
bounds their tests use (not collected as a test module)."""
import numpy as np
import torch

# One rounding to nearest with p significant bits is at most 2^-p relative:
# bf16 has 8 of them (torch.finfo(bf16).eps is 2^-7, twice that), fp32 24.
U_BF16 = torch.finfo(torch.bfloat16).eps / 2
U_F32 = torch.finfo(torch.float32).eps / 2


def bank(gen, groups, rows, cols, group):
    """(codes [G, rows, cols / 2] uint8, scales [G, rows, cols / group] bf16) on
    the CPU: every code, scales of both signs over a factor of eight."""
    q = torch.randint(0, 256, (groups, rows, cols // 2), generator=gen, dtype=torch.uint8)
    e = torch.rand((groups, rows, cols // group), generator=gen) * 3 - 8
    sign = torch.randint(0, 2, e.shape, generator=gen) * 2 - 1
    return q, (sign * torch.exp2(e)).bfloat16()


def dequant64(q, s):
    """fp64 weights [rows, cols] of one group's codes and scales."""
    q, s = q.cpu().numpy(), s.float().cpu().numpy().astype(np.float64)
    w = np.empty((q.shape[0], 2 * q.shape[1]))
    w[:, 0::2] = (q & 15).astype(np.float64) - 8
    w[:, 1::2] = (q >> 4).astype(np.float64) - 8
    return w * np.repeat(s, w.shape[1] // s.shape[1], axis=1)


def fp8_rows(x):
    """E4M3 codes (uint8) and fp32 scales per 128 columns of fp32 rows x."""
    m = x.view(x.shape[0], -1, 128)
    s = (m.abs().amax(-1) / 448.0).clamp_min(1e-30)
    q = (m / s[..., None]).to(torch.float8_e4m3fn)
    return q.view(x.shape).view(torch.uint8), s


def values64(x, xs=None):
    """fp64 values of bf16 rows, or of E4M3 codes with their scales."""
    if xs is None:
        return x.float().cpu().numpy().astype(np.float64)
    v = x.cpu().view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    return v * np.repeat(xs.cpu().numpy().astype(np.float64), 128, axis=1)


def dot_bound(w, x):
    """Bound on the fp32 error of x w^T, elementwise: the products are exact
    in fp32; a tensor-core step adds 16 of them, each aligned to the largest
    (at most 2^-23 of it lost per term), and the steps of K columns, their
    group scales and the row scales are K / 16 + 8 further fp32 operations,
    each 2^-23 of at most the sum of magnitudes."""
    n = w.shape[1] / 16 + 8 + 16
    return n * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)


def silu(g):
    return g / (1 + np.exp(-np.clip(g, -700, None)))


def swiglu64(x, gu, dn):
    """(y, bound) of one expert for rows x: W_down (SiLU(W_gate x) * W_up x),
    and the error of a kernel that keeps the two products in fp32, takes SiLU
    with the fast exponential and division (2^-20 relative), rounds H to bf16
    and sums the second product in fp32."""
    F = gu.shape[0] // 2
    z, dz = x @ gu.T, dot_bound(gu, x)
    g, u, dg, du = z[:, :F], z[:, F:], dz[:, :F], dz[:, F:]
    h = silu(g) * u
    # |SiLU'| <= 1.1
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + (U_BF16 + 2.0 ** -20) * np.abs(h)
    dh += U_BF16 * dh
    y = h @ dn.T
    return y, dh @ np.abs(dn).T + dot_bound(dn, np.abs(h) + dh)


def close(got, ref, bound, rounding=U_BF16):
    """Every element within its bound and one rounding to the output's type."""
    got = got.float().cpu().numpy().astype(np.float64)
    lim = bound + rounding * (np.abs(ref) + bound) * 1.001 + 1e-38
    bad = ~(np.abs(got - ref) <= lim)
    if bad.any():
        at = np.argwhere(bad)[0]
        raise AssertionError(f"{int(bad.sum())} of {bad.size} outside; first at {tuple(at)}: got "
                             f"{got[tuple(at)]}, want {ref[tuple(at)]} +- {lim[tuple(at)]}")
