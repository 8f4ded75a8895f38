"""One MoE block of a decode step with 4-bit expert weights, on seeded
synthetic inputs: the residual sum and RMS norm, the router on the norm's bf16
rows, the routed and shared experts on its 8-bit rows (or its bf16 rows), and
the weighted combine; with --L also the latent projections in 4 bits around
the routed experts.

    python -m fine_grained_sparse_gb300.run_decode --T 8 --E 64 --K 8
    python -m fine_grained_sparse_gb300.run_decode --T 4 --E 64 --K 8 --L 3584 --bf16-rows

Prints the device time of the block; --check compares it with a plain fp32
torch form of every step.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import synth  # noqa: E402

import fine_grained_sparse_gb300 as fgs  # noqa: E402

EPS = 1e-6


def random_bank(gen, groups, rows, cols, group):
    """4-bit codes and scales of weights of about N(0, 0.02)'s size."""
    q = torch.randint(0, 256, (groups, rows, cols // 2), generator=gen, device="cuda",
                      dtype=torch.uint8)
    s = torch.rand((groups, rows, cols // group), generator=gen, device="cuda") + 0.5
    return q, s.mul_(0.02 / 4.6).bfloat16()


class Block:
    """The weights of one block, packed once, and its buffers for T rows."""

    def __init__(self, shape, T, group=32, rows8=True, seed=0, keep=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.shape, self.T, self.group, self.rows8 = shape, T, group, rows8
        d, E, S, L = shape.d_model, shape.E_routed, shape.E_shared, shape.d_latent
        de, F, Fs = shape.d_expert, shape.d_ff, shape.d_ff_shared
        self.cfg = fgs.config(shape, weight_layout=fgs.MOE_WEIGHTS_PACKED_INT4_G32 if group == 32
                              else fgs.MOE_WEIGHTS_PACKED_INT4_G128)
        dims = {"gate_up": (0, E, 2 * F, de), "down": (1, E, de, F)}
        if S:
            dims.update(s_gate_up=(0, S, 2 * Fs, d), s_down=(1, S, d, Fs))
        if L:
            dims.update(lat_down=(1, 1, L, d), lat_up=(1, 1, d, L))
        self.raw, self.w = {}, {}
        for name, (kind, n, rows, cols) in dims.items():
            q, s = random_bank(g, n, rows, cols, group)
            self.w[name] = fgs.pack_int4(kind, q, s)
            if keep:
                self.raw[name] = (q, s)
        self.W_r, self.bias = synth.router_params(shape, "cuda", seed)
        self.norm_w = (1 + 0.1 * torch.randn((d,), generator=g, device="cuda")).bfloat16()
        bf = dict(dtype=torch.bfloat16, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        K = shape.K
        self.h, self.x = torch.empty((T, d), **bf), torch.empty((T, d), **bf)
        self.x8 = torch.empty((T, d), dtype=torch.float8_e4m3fn, device="cuda")
        self.xs = torch.empty((T, d // 128), device="cuda")
        self.idx, self.topk_w = torch.empty((T, K), **i32), torch.empty((T, K), device="cuda")
        self.counts, self.offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        self.perm, self.inv = torch.empty(T * K, **i32), torch.empty(T * K, **i32)
        self.Y = torch.empty((T * K, de), **bf)
        self.Ysh = torch.empty((S, T, d), **bf) if S else None
        self.y, self.lat, self.r = (torch.empty((T, n), **bf) for n in (d, max(L, 1), max(L, 1)))
        self.nws = fgs.moe_workspace_size(self.cfg, T)
        self.ws = torch.zeros(self.nws, dtype=torch.uint8, device="cuda")

    def __call__(self, attn_out, residual):
        """(h, y): the new residual stream and the block's output."""
        c, T, w, s = self.cfg, self.T, self.w, self.shape
        d, L, S = s.d_model, s.d_latent, s.E_shared
        fgs.moe_add_rmsnorm(fgs.MOE_BF16, T, d, attn_out, residual, self.norm_w, EPS, self.h,
                            self.x, self.x8, self.xs)
        fgs.moe_router(c, T, self.x, self.W_r, self.bias, self.idx, self.topk_w, self.ws, self.nws)
        fgs.moe_permute(c, T, self.idx, self.counts, self.offsets, self.perm, self.inv, self.ws,
                        self.nws)
        rows, scale = (self.x8, self.xs) if self.rows8 else (self.x, None)
        xe = rows
        if L:  # the latent rows are bf16: an 8-bit form of them is not the norm's to make
            fgs.moe_linear_int4(T, d, L, self.group, rows, scale, w["lat_down"], None, self.lat)
            xe = self.lat
        shared = (w.get("s_gate_up"), w.get("s_down"), self.Y, self.Ysh, self.ws, self.nws)
        if self.rows8 and not L:
            fgs.moe_grouped_swiglu_fp8_rows(c, T, xe, scale, self.offsets, self.perm, None,
                                            w["gate_up"], w["down"], rows if S else None,
                                            scale if S else None, *shared)
        else:
            fgs.moe_grouped_swiglu(c, T, xe, self.offsets, self.perm, None, w["gate_up"],
                                   w["down"], self.x if S else None, *shared)
        if not L:
            fgs.moe_combine(c, T, self.Y, self.inv, self.topk_w, self.Ysh, self.y)
        else:
            fgs.moe_combine(c, T, self.Y, self.inv, self.topk_w, None, self.r)
            add = self.Ysh[0] if S else None
            fgs.moe_linear_int4(T, L, d, self.group, self.r, None, w["lat_up"], add, self.y)
            for i in range(1, S):
                self.y += self.Ysh[i]
        return self.h, self.y


def plain_block(b: Block, attn_out, residual):
    """The same step in elementary fp32 torch operations, given the block's
    routing (near-equal router scores may order differently)."""
    def weights(name, i):
        q, s = (t[i] for t in b.raw[name])
        v = torch.stack((q & 15, q >> 4), -1).view(q.shape[0], s.shape[1], -1).float() - 8
        return (v * s.float()[..., None]).view(q.shape[0], -1)

    def expert(u, gu, dn):
        g, v = (u @ gu.t()).chunk(2, 1)
        return (torch.nn.functional.silu(g) * v) @ dn.t()

    h = attn_out.float() + residual.float()
    x = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * b.norm_w.float()
    s = b.shape
    xe = x @ weights("lat_down", 0).t() if s.d_latent else x
    out = torch.zeros_like(xe)
    idx = b.idx.long()
    for e in idx.unique().tolist():
        t, k = (idx == e).nonzero(as_tuple=True)
        y = expert(xe[t], weights("gate_up", e), weights("down", e))
        out.index_add_(0, t, y * b.topk_w[t, k][:, None])
    if s.d_latent:
        out = out @ weights("lat_up", 0).t()
    for i in range(s.E_shared):
        out = out + expert(x, weights("s_gate_up", i), weights("s_down", i))
    return h, out


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--T", type=int, default=8)
    ap.add_argument("--d", type=int, default=7168)
    ap.add_argument("--E", type=int, default=64)
    ap.add_argument("--K", type=int, default=8)
    ap.add_argument("--F", type=int, default=2048)
    ap.add_argument("--S", type=int, default=1)
    ap.add_argument("--L", type=int, default=0)
    ap.add_argument("--group", type=int, default=32, choices=(32, 128))
    ap.add_argument("--bf16-rows", action="store_true", help="experts read bf16 rows, not 8-bit")
    ap.add_argument("--iters", type=int, default=20)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    shape = synth.custom(name="decode_block", T=a.T, d_model=a.d, E_routed=a.E, K=a.K,
                         E_shared=a.S, d_ff=a.F, d_ff_shared=a.F, d_latent=a.L)
    b = Block(shape, a.T, a.group, not a.bf16_rows, keep=a.check)
    g = torch.Generator(device="cuda").manual_seed(1)
    attn, res = (torch.randn((a.T, a.d), generator=g, device="cuda").bfloat16() for _ in range(2))
    for _ in range(3):
        b(attn, res)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for _ in range(a.iters):
        b(attn, res)
    stop.record()
    torch.cuda.synchronize()
    status = fgs.moe_get_device_status(b.ws) or fgs.moe_get_device_status(fgs.moe_status_word())
    if status:
        raise SystemExit("device status: " + fgs.moe_status_string(status))
    print(f"block of {a.T} tokens: {start.elapsed_time(stop) / a.iters * 1e3:.1f} us")
    if a.check:
        h, y = plain_block(b, attn, res)
        rel = lambda p, q: float((p.float() - q).norm() / q.norm())  # noqa: E731
        print(f"relative difference to the plain form: h {rel(b.h, h):.2e}, y {rel(b.y, y):.2e}")


if __name__ == "__main__":
    main()
