"""The measured cases of the training operators around the experts' products:
the rows in expert order (``moe_gather``), the gradients of the weighted combine
(``moe_combine_backward``) and of the gate weights (``moe_router_backward``), the
residual sum with its layer norm (``moe_add_layernorm``), the gradients of both
norms (``moe_norm_backward``) and the AdamW step over many tensors
(``moe_adamw``).

With ``own`` false ``run`` computes an operator in elementary torch operations
in fp32, rounded once at the end; with ``own`` true it makes the library's
calls.  AdamW's 8-bit states are E4M3 codes with one fp32 scale for 128
elements: the first moment rounded to nearest, the root of the second moment
rounded up or down at random, 16 bits of a hash of the element's place deciding.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128  # elements of a state that share one scale
EPS = 1e-6
SCALING = 2.827
ADAM = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8}
M32 = 0xFFFFFFFF


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one token to its experts' rows: latency
        {"name": "gather T1 K8 d7168", "op": "gather", "T": 1, "K": 8, "E": 384, "d": 7168,
         "dtype": "bf16", "weights": True, "bad": 0.0},
        # the layer's training batch into expert order: bandwidth
        {"name": "gather T8192 K8 d7168", "op": "gather", "T": 8192, "K": 8, "E": 384, "d": 7168,
         "dtype": "bf16", "weights": True, "bad": 0.0},
        # fp32 rows of a ragged batch on the way back, some pairs rejected by the sort
        {"name": "combine back T301 K6 d1920 f32", "op": "combine_bwd", "T": 301, "K": 6, "E": 64,
         "d": 1920, "dtype": "f32", "weights": True, "bad": 0.02},
        # the latent form's batch on the way back
        {"name": "combine back T4096 K16 d3584", "op": "combine_bwd", "T": 4096, "K": 16, "E": 896,
         "d": 3584, "dtype": "bf16", "weights": True, "bad": 0.0},
        # the router's gradient for a small batch: latency
        {"name": "router back T128 E384 K8", "op": "router_bwd", "T": 128, "E": 384, "K": 8,
         "renorm": True, "bad": 0.0},
        # and for the latent form's experts at the training batch
        {"name": "router back T8192 E896 K16", "op": "router_bwd", "T": 8192, "E": 896, "K": 16,
         "renorm": True, "bad": 0.0},
        # a few rows before the layer, with the residual stream
        {"name": "layernorm T33 d7168", "op": "layernorm", "T": 33, "d": 7168, "dtype": "bf16",
         "residual": True, "bias": True},
        # fp32 rows of an odd count, bandwidth
        {"name": "layernorm T8191 d3584 f32", "op": "layernorm", "T": 8191, "d": 3584,
         "dtype": "f32", "residual": False, "bias": True},
        # the way back through a layer norm whose width no power of two divides
        {"name": "layernorm back T777 d1000 f32", "op": "norm_bwd", "kind": "layer", "T": 777,
         "d": 1000, "dtype": "f32", "dh": False, "dw": True},
        # the way back through the norm before the layer at the training batch
        {"name": "rmsnorm back T8192 d7168", "op": "norm_bwd", "kind": "rms", "T": 8192, "d": 7168,
         "dtype": "bf16", "dh": True, "dw": True},
        # norm weights and router biases of all blocks in one step: many small tensors
        {"name": "adamw 182 small f32", "op": "adamw", "sizes": "7168x122,384x60", "param": "f32",
         "grad": "f32", "master": False, "bits": 32, "step": 7},
        # the banks of a few experts in bf16 with an fp32 master copy, states in 8 bits
        {"name": "adamw 352M bf16 states8", "op": "adamw", "sizes": "234881024x1,117440512x1",
         "param": "bf16", "grad": "bf16", "master": True, "bits": 8, "step": 1000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gather", "combine_bwd", "router_bwd", "layernorm", "norm_bwd", "norm_bwd",
                     "adamw", "adamw"])
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    if op in ("gather", "combine_bwd"):
        d = 128 * _log(rng, 1, 56) if dtype == "bf16" else 32 * _log(rng, 1, 112)
        K = rng.choice([1, 2, 4, 6, 8, 16])
        most = 8192 * 8 * 7168 * 2 if op == "gather" else 4096 * 16 * 3584 * 2
        T = min(_log(rng, 1, 8192), most // (K * d * (2 if dtype == "bf16" else 4)))
        return {"op": op, "T": max(1, T), "K": K, "E": rng.choice([16, 63, 64, 384, 896]), "d": d,
                "dtype": dtype, "weights": rng.random() < 0.7,
                "bad": 0.05 if rng.random() < 0.3 else 0.0}
    if op == "router_bwd":
        return {"op": op, "T": _log(rng, 1, 8192), "E": rng.randint(16, 896),
                "K": rng.choice([1, 2, 4, 6, 8, 16]), "renorm": rng.random() < 0.8,
                "bad": 0.05 if rng.random() < 0.3 else 0.0}
    if op in ("layernorm", "norm_bwd"):
        d = 8 * _log(rng, 8, 1024) if rng.random() < 0.7 else _log(rng, 64, 8192)
        b = 2 if dtype == "bf16" else 4
        T = max(1, min(_log(rng, 1, 8192), 8192 * 7168 * 2 // (d * b)))
        if op == "layernorm":
            return {"op": op, "T": T, "d": d, "dtype": dtype, "residual": rng.random() < 0.6,
                    "bias": rng.random() < 0.7}
        return {"op": op, "kind": rng.choice(["rms", "layer"]), "T": T, "d": d, "dtype": dtype,
                "dh": rng.random() < 0.6, "dw": rng.random() < 0.85}
    kinds = rng.randint(1, 3)
    sizes = []
    for _ in range(kinds):
        n = _log(rng, 1, 60_000_000)
        sizes.append(f"{n}x{max(1, min(_log(rng, 1, 150), 100_000_000 // n))}")
    param = "bf16" if rng.random() < 0.6 else "f32"
    return {"op": "adamw", "sizes": ",".join(sizes), "param": param,
            "grad": "bf16" if param == "bf16" and rng.random() < 0.7 else "f32",
            "master": param == "bf16" and rng.random() < 0.6, "bits": rng.choice([8, 32]),
            "step": _log(rng, 1, 20000)}


def _sizes(case):
    """The element counts of an AdamW case's tensors, one after the other."""
    return [int(n) for part in case["sizes"].split(",") for n in [part.split("x")[0]]
            for _ in range(int(part.split("x")[1]))]


def work(case):
    c = case
    b = 2 if c.get("dtype") == "bf16" else 4
    if c["op"] == "router_bwd":
        T, K = c["T"], c["K"]
        return {"bytes": 4 * T * c["E"] + 12 * T * K, "flops": 12 * T * K}
    if c["op"] in ("gather", "combine_bwd"):
        T, K, d = c["T"], c["K"], c["d"]
        if c["op"] == "gather":
            n = T * d * b + T * K * d * b + 4 * T * K + 8 * T * K * c["weights"]
            return {"bytes": n, "flops": 0}
        n = T * d * b + 2 * T * K * d * b + 8 * T * K + 4 * T * K * c["weights"]
        return {"bytes": n, "flops": 3 * T * K * d}
    if c["op"] == "layernorm":
        n = c["T"] * c["d"] * b * (2 + 2 * c["residual"]) + c["d"] * b * (1 + c["bias"])
        return {"bytes": n, "flops": 8 * c["T"] * c["d"]}
    if c["op"] == "norm_bwd":
        n = c["T"] * c["d"] * b * (3 + c["dh"]) + c["d"] * b
        n += 4 * c["d"] * c["dw"] * (1 + (c["kind"] == "layer"))
        return {"bytes": n, "flops": 14 * c["T"] * c["d"]}
    n = sum(_sizes(c))
    each = (4 if c["param"] == "bf16" and not c["master"] else 2 if c["master"] else 8)
    each += (2 if c["grad"] == "bf16" else 4) + 8 * c["master"]
    each += 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": int(n * each), "flops": 20 * n}


# --------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 29)


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _routing(g, T, K, E, bad):
    """Distinct experts of every token, popularities a factor of ten apart;
    some indices outside [0, E) when ``bad`` is set."""
    popular = torch.rand((E,), generator=g, device="cuda") * math.log(10.0)
    noise = torch.rand((T, E), generator=g, device="cuda").clamp_min_(1e-9)
    gumbel = -torch.log((-torch.log(noise)).clamp_min_(1e-9))
    idx = (popular + gumbel).topk(K, dim=1).indices
    if bad:
        idx[torch.rand((T, K), generator=g, device="cuda") < bad] = E
    return idx.to(torch.int32)


def _slots(idx, E):
    """The sort of the pairs by expert: (perm, inv, pairs kept)."""
    flat = idx.reshape(-1)
    perm = torch.sort(flat, stable=True).indices
    kept = int((flat < E).sum())
    inv = torch.empty_like(flat)
    inv[perm] = torch.arange(flat.numel(), device="cuda", dtype=torch.int32)
    inv[flat >= E] = -1
    return perm.to(torch.int32), inv, kept


def _mix64(x):
    """The finaliser of splitmix64."""
    x = (x + 0x9E3779B97F4A7C15) & (2 ** 64 - 1)
    x = ((x ^ (x >> 30)) * 0xBF58476D1CE4E5B9) & (2 ** 64 - 1)
    x = ((x ^ (x >> 27)) * 0x94D049BB133111EB) & (2 ** 64 - 1)
    return x ^ (x >> 31)


def _quantised(x):
    """E4M3 codes and scales of fp32 values, 128 to a scale, to nearest."""
    s = x.abs().amax(1) * (1.0 / E4M3_MAX)
    q = torch.where(s[:, None] > 0, x / s[:, None], torch.zeros_like(x))
    return q.to(torch.float8_e4m3fn), s


def _prepare_adamw(c, g, st, seed):
    """All tensors of the step in one buffer a kind, every tensor beginning on
    a block of 128 elements; what lies behind a tensor's end stays 0."""
    sizes = _sizes(c)
    blocks = [-(-n // BLOCK) for n in sizes]
    first = [0]
    for b in blocks:
        first.append(first[-1] + b)
    total = first[-1]
    count = torch.tensor(blocks, device="cuda")
    which = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), count)
    begin = torch.tensor(first[:-1], device="cuda")[which]
    st["index"] = (torch.arange(total, device="cuda") - begin) * BLOCK  # of a block's first element
    left = torch.tensor(sizes, device="cuda")[which] - st["index"]
    keys = [_mix64(int(seed) + 0x9E3779B97F4A7C15 * k & 2 ** 64 - 1) >> 32 for k in range(len(sizes))]
    st["key"] = torch.tensor(keys, device="cuda")[which]
    decays = [0.1 if k % 2 == 0 else 0.0 for k in range(len(sizes))]  # every other without decay
    factor = [1.0 - ADAM["lr"] * w for w in decays]
    st["factor"] = torch.tensor(factor, device="cuda", dtype=torch.float32)[which]
    st["factor64"] = torch.tensor(factor, device="cuda", dtype=torch.float64)[which]
    inside = torch.arange(BLOCK, device="cuda") < left[:, None]
    level = torch.exp(1.5 * _rand(g, total, 1))  # gradients' sizes differ from block to block
    p = _rand(g, total, BLOCK).mul_(0.02).mul_(inside)
    st["g"] = (_rand(g, total, BLOCK) * level * 1e-3).mul_(inside).to(_dtype(c["grad"]))
    m = (_rand(g, total, BLOCK) * level * 2e-4).mul_(inside)
    r = ((_rand(g, total, BLOCK).abs_() + 0.3) * level * 1e-3).mul_(inside)
    if c["bits"] == 8:
        st["m"], st["ms"] = _quantised(m)
        st["v"], st["vs"] = _quantised(r)
    else:
        st["m"], st["v"] = m, r.square_()
    if c["master"]:
        st["master"] = p
    st["p"] = p.to(_dtype(c["param"])) if c["param"] == "bf16" else p
    # a device scalar, as a clip of the gradients' norm leaves it
    st["gs"] = torch.full((1,), 0.75, device="cuda")
    st["seed"] = int(seed)
    if own:
        import fine_grained_sparse_gb300 as fgs
        flat = {k: st[k].view(-1) for k in ("p", "g", "m", "v", "master") if k in st}
        st["table"] = fgs.adamw_table([
            {"param": flat["p"][BLOCK * f:], "grad": flat["g"][BLOCK * f:],
             "exp_avg": flat["m"][BLOCK * f:], "exp_avg_sq": flat["v"][BLOCK * f:],
             "master": flat["master"][BLOCK * f:] if c["master"] else None,
             "exp_avg_scale": st["ms"][f:] if c["bits"] == 8 else None,
             "exp_avg_sq_scale": st["vs"][f:] if c["bits"] == 8 else None,
             "n": n, "weight_decay": w} for f, n, w in zip(first, sizes, decays)])


def prepare(case, seed):
    g = _generator(seed)
    c, st = case, {"case": dict(case)}
    if own:
        import fine_grained_sparse_gb300 as fgs
        st["fgs"] = fgs
    if c["op"] == "adamw":
        _prepare_adamw(c, g, st, seed)
        return st
    T = c["T"]
    if c["op"] in ("gather", "combine_bwd", "router_bwd"):
        K, E = c["K"], c["E"]
        st["idx"] = _routing(g, T, K, E, c["bad"])
        if own:
            d = c.get("d", 128)
            st["cfg"] = fgs.config(d_model=d, d_ff=64, E_routed=E, K=K,
                                   dtype=fgs.MOE_F32 if c.get("dtype") == "f32" else fgs.MOE_BF16,
                                   norm_topk_prob=c.get("renorm", True),
                                   routed_scaling_factor=SCALING)
    if c["op"] == "router_bwd":
        st["z"] = 1.5 * _rand(g, T, E)
        st["dw"] = _rand(g, T, K)
        if own:
            st["dz"] = torch.empty((T, E), device="cuda")
        return st
    dt = _dtype(c["dtype"])
    if c["op"] in ("gather", "combine_bwd"):
        d = c["d"]
        st["perm"], st["inv"], st["kept"] = _slots(st["idx"], E)
        if c["weights"]:
            w = torch.rand((T, K), generator=g, device="cuda") + 0.05
            st["w"] = SCALING * w / w.sum(1, keepdim=True)
        # rows behind the last pair stay as they were
        rows = torch.zeros((T * K, d), dtype=dt, device="cuda")
        if c["op"] == "gather":
            st["x"] = _rand(g, T, d).to(dt)
            st["xp"] = rows
            if c["weights"]:
                st["wp"] = torch.zeros((T * K,), device="cuda")
        else:
            st["dy"] = _rand(g, T, d).to(dt)
            st["Y"] = _rand(g, T * K, d).mul_(0.3).to(dt)
            st["dY"] = rows
            if own:
                st["dw"] = torch.empty((T, K), device="cuda")
        return st
    d = c["d"]
    st["w"] = (1.0 + 0.2 * _rand(g, d)).to(dt)
    st["x"] = (2.0 * _rand(g, T, d) + 0.5 * _rand(g, T, 1)).to(dt)
    if c["op"] == "layernorm":
        if c["residual"]:
            st["r"] = (3.0 * _rand(g, T, d)).to(dt)
        if c["bias"]:
            st["b"] = (0.1 * _rand(g, d)).to(dt)
        if own:
            st["h"] = torch.empty_like(st["x"]) if c["residual"] else None
            st["y"] = torch.empty_like(st["x"])
        return st
    st["dy"] = _rand(g, T, d).to(dt)
    if c["dh"]:
        st["dh"] = _rand(g, T, d).to(dt)
    if own:
        st["dx"] = torch.empty_like(st["x"])
        if c["dw"]:
            st["dw"] = torch.empty((d,), device="cuda")
            st["nws"] = fgs.moe_norm_backward_workspace_size(T, d)
            st["ws"] = torch.zeros(st["nws"], dtype=torch.uint8, device="cuda")
            if c["kind"] == "layer":
                st["db"] = torch.empty((d,), device="cuda")
    return st


# -------------------------------------------------------------- the two forms
def run(state):
    op = state["case"]["op"]
    if own:
        return {"gather": _own_gather, "combine_bwd": _own_combine_bwd,
                "router_bwd": _own_router_bwd, "layernorm": _own_layernorm,
                "norm_bwd": _own_norm_bwd, "adamw": _own_adamw}[op](state)
    return {"gather": _plain_gather, "combine_bwd": _plain_combine_bwd,
            "router_bwd": _plain_router_bwd, "layernorm": _plain_layernorm,
            "norm_bwd": _plain_norm_bwd, "adamw": _plain_adamw}[op](state)


def _own_gather(s):
    s["fgs"].moe_gather(s["cfg"], s["case"]["T"], s["x"], s["inv"], s.get("w"), s["xp"],
                        s.get("wp"))
    return {"xp": s["xp"], "wp": s.get("wp")}


def _plain_gather(s):
    pairs = s["perm"][:s["kept"]].long()
    s["xp"][:s["kept"]] = s["x"][pairs // s["case"]["K"]]
    if "w" in s:
        s["wp"][:s["kept"]] = s["w"].view(-1)[pairs]
    return {"xp": s["xp"], "wp": s.get("wp")}


def _own_combine_bwd(s):
    s["fgs"].moe_combine_backward(s["cfg"], s["case"]["T"], s["dy"], s["Y"], s["inv"], s.get("w"),
                                  s["dY"], s["dw"])
    return {"dY": s["dY"], "dw": s["dw"]}


def _plain_combine_bwd(s):
    c = s["case"]
    pairs = s["perm"][:s["kept"]].long()
    dy = s["dy"].float()[pairs // c["K"]]
    dw = torch.zeros((c["T"] * c["K"],), device="cuda")
    dw[pairs] = (s["Y"][:s["kept"]].float() * dy).sum(1)
    if "w" in s:
        dy = dy * s["w"].view(-1)[pairs][:, None]
    s["dY"][:s["kept"]] = dy.to(s["dY"].dtype)
    return {"dY": s["dY"], "dw": dw.view(c["T"], c["K"])}


def _own_router_bwd(s):
    s["fgs"].moe_router_backward(s["cfg"], s["case"]["T"], s["z"], s["idx"], s["dw"], s["dz"])
    return {"dz": s["dz"]}


def _plain_router_bwd(s):
    c = s["case"]
    kept = s["idx"] < c["E"]
    at = torch.where(kept, s["idx"], 0).long()
    z = s["z"].gather(1, at)
    p = torch.where(kept, 1.0 / (1.0 + torch.exp(-z)), 0.0)
    dw = torch.where(kept, s["dw"], 0.0)
    if c["renorm"] and c["K"] > 1:
        p = p / (p.sum(1, keepdim=True) + 1e-20)
        dw = dw - (dw * p).sum(1, keepdim=True)
    dz = SCALING * p * dw / (1.0 + torch.exp(z))
    return {"dz": torch.zeros_like(s["z"]).scatter_add_(1, at, dz)}


def _own_layernorm(s):
    c, fgs = s["case"], s["fgs"]
    fgs.moe_add_layernorm(fgs.MOE_BF16 if c["dtype"] == "bf16" else fgs.MOE_F32, c["T"], c["d"],
                          s["x"], s.get("r"), s["w"], s.get("b"), EPS, s["h"], s["y"])
    return {"h": s["h"], "y": s["y"]}


def _plain_layernorm(s):
    v, out = s["x"].float(), {}
    if "r" in s:
        v = v + s["r"].float()
        out["h"] = v.to(s["x"].dtype)
    v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    if "b" in s:
        v = v + s["b"].float()
    out["y"] = v.to(s["x"].dtype)
    return out


def _own_norm_bwd(s):
    c, fgs = s["case"], s["fgs"]
    kind = fgs.MOE_NORM_RMS if c["kind"] == "rms" else fgs.MOE_NORM_LAYER
    fgs.moe_norm_backward(kind, fgs.MOE_BF16 if c["dtype"] == "bf16" else fgs.MOE_F32, c["T"],
                          c["d"], s["x"], None, s["w"], EPS, s["dy"], s.get("dh"), s["dx"],
                          s.get("dw"), s.get("db"), s.get("ws"), s.get("nws", 0))
    return {"dx": s["dx"], "dw": s.get("dw"), "db": s.get("db")}


def _plain_norm_bwd(s):
    c, out = s["case"], {}
    v, dy = s["x"].float(), s["dy"].float()
    if c["kind"] == "layer":
        v = v - v.mean(1, keepdim=True)
    r = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    v = v * r
    if c["dw"]:
        out["dw"] = (dy * v).sum(0)
        if c["kind"] == "layer":
            out["db"] = dy.sum(0)
    g = dy * s["w"].float()
    dx = g - v * (g * v).mean(1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * r
    if c["dh"]:
        dx = dx + s["dh"].float()
    out["dx"] = dx.to(s["x"].dtype)
    return out


def _own_adamw(s):
    c, fgs = s["case"], s["fgs"]
    kinds = {"bf16": fgs.MOE_BF16, "f32": fgs.MOE_F32}
    fgs.moe_adamw(s["table"], kinds[c["param"]], kinds[c["grad"]], c["bits"], ADAM["lr"],
                  ADAM["beta1"], ADAM["beta2"], ADAM["eps"], c["step"], s["gs"], s["seed"])
    return {k: s[k] for k in ("p", "master", "m", "ms", "v", "vs") if k in s}


def _noise(s):
    """16 random bits of every element, in [0, 65536): of the hash of its
    pair's number, the low half for the even element."""
    pair = (s["index"] // 2)[:, None] + torch.arange(BLOCK // 2, device="cuda")
    h = (pair & M32) ^ s["key"][:, None] ^ ((pair >> 32) * 0x9E3779B9 & M32)
    h = (h ^ h >> 16) * 0x85EBCA6B & M32  # the finaliser of MurmurHash3
    h = (h ^ h >> 13) * 0xC2B2AE35 & M32
    h = (h ^ h >> 16).to(torch.int64)
    return torch.stack((h & 0xFFFF, h >> 16), -1).view(h.shape[0], BLOCK).to(torch.int32)


def _plain_adamw(s):
    c, a = s["case"], ADAM
    g = s["g"].float() * s["gs"]
    if c["bits"] == 8:
        m = s["m"].float() * s["ms"][:, None]
        v = s["v"].float() * s["vs"][:, None]
        v = v * v
    else:
        m, v = s["m"], s["v"]
    m = m * a["beta1"] + g * (1.0 - a["beta1"])
    v = v * a["beta2"] + g * g * (1.0 - a["beta2"])
    r = torch.sqrt(v)
    size = a["lr"] / (1.0 - a["beta1"] ** c["step"])
    root = 1.0 / math.sqrt(1.0 - a["beta2"] ** c["step"])
    p = s["master"] if c["master"] else s["p"].float()
    p = p * s["factor"][:, None] - m / (r * root + a["eps"]) * size
    if c["master"]:
        s["master"].copy_(p)
    s["p"].copy_(p)
    if c["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {k: s[k] for k in ("p", "master", "m", "v") if k in s}
    q, scale = _quantised(m)
    s["m"].copy_(q)
    s["ms"].copy_(scale)
    scale = r.amax(1) * (1.0 / E4M3_MAX)
    q = torch.where(scale[:, None] > 0, r / scale[:, None], torch.zeros_like(r))
    u = _noise(s)
    # below 2^-6 the codes are 2^-9 apart, above it a mantissa's three bits
    low = torch.floor(q * 512.0 + (u.float() + 0.5) * 2.0 ** -16).to(torch.int32)
    high = (q.view(torch.int32) + (u << 4) + 8 >> 20) - (120 << 3)
    code = torch.where(q < 2.0 ** -6, low, high).clamp(0, 0x7E)
    code = torch.where((code == 0) & (r > 0), 1, code)
    s["v"].view(torch.uint8).copy_(code)
    s["vs"].copy_(scale)
    return {k: s[k] for k in ("p", "master", "m", "ms", "v", "vs") if k in s}


# -------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """What ``run`` returns from the definitions in fp64 (None for the 8-bit
    codes' place: their scale's last bit decides some of them)."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, f = case, torch.float64
    if c["op"] == "adamw":
        return _exact_adamw(s)
    if c["op"] == "gather":
        n, flat = c["T"] * c["K"], s["inv"].long()
        xp = torch.zeros((n + 1, c["d"]), dtype=f, device="cuda")
        xp[torch.where(flat < 0, n, flat)] = s["x"].to(f).repeat_interleave(c["K"], 0)
        wp = None
        if c["weights"]:
            wp = torch.zeros((n + 1,), dtype=f, device="cuda")
            wp[torch.where(flat < 0, n, flat)] = s["w"].to(f).flatten()
            wp = wp[:n]
        return {"xp": xp[:n], "wp": wp}
    if c["op"] == "combine_bwd":
        n, dY = c["T"] * c["K"], torch.zeros(s["dY"].shape, dtype=f, device="cuda")
        dw = torch.zeros((c["T"], c["K"]), dtype=f, device="cuda")
        inv = s["inv"].view(c["T"], c["K"]).long()
        for k in range(c["K"]):
            t = (inv[:, k] >= 0).nonzero()[:, 0]
            dy, slot = s["dy"].to(f)[t], inv[t, k]
            dw[t, k] = torch.linalg.vecdot(s["Y"][slot].to(f), dy)
            dY[slot] = dy * s["w"][t, k].to(f)[:, None] if c["weights"] else dy
        return {"dY": dY, "dw": dw}
    if c["op"] == "router_bwd":
        z = s["z"].to(f).requires_grad_()
        kept = s["idx"] < c["E"]
        sel = torch.sigmoid(torch.take_along_dim(z, s["idx"].long().clamp(max=c["E"] - 1), 1)) * kept
        w = sel / (sel.sum(1, keepdim=True) + 1e-20) if c["renorm"] and c["K"] > 1 else sel
        (SCALING * w * s["dw"].to(f)).sum().backward()
        return {"dz": z.grad}
    if c["op"] == "layernorm":
        h = s["x"].to(f) + (s["r"].to(f) if c["residual"] else 0.0)
        var, mu = torch.var_mean(h, 1, correction=0, keepdim=True)
        y = (h - mu) / torch.sqrt(var + EPS) * s["w"].to(f) + (s["b"].to(f) if c["bias"] else 0.0)
        return {"h": h, "y": y} if c["residual"] else {"y": y}
    x = s["x"].to(f).requires_grad_()
    w = s["w"].to(f).requires_grad_()
    b = torch.zeros(c["d"], dtype=f, device="cuda", requires_grad=True)
    if c["kind"] == "rms":
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / c["d"] + EPS) * w
    else:
        var, mu = torch.var_mean(x, 1, correction=0, keepdim=True)
        y = (x - mu) / torch.sqrt(var + EPS) * w + b
    y.backward(s["dy"].to(f))
    out = {"dx": x.grad + (s["dh"].to(f) if c["dh"] else 0.0)}
    if c["dw"]:
        out["dw"] = w.grad
        if c["kind"] == "layer":
            out["db"] = b.grad
    return out


def _exact_adamw(s):
    c, f, a = s["case"], torch.float64, ADAM
    g = s["g"].to(f) * float(s["gs"])
    if c["bits"] == 8:
        m, v = (s[k].to(torch.float32).to(f) * s[k + "s"].to(f)[:, None] for k in ("m", "v"))
        v = v.square_()
    else:
        m, v = s["m"].to(f), s["v"].to(f)
    m = torch.lerp(g, m, a["beta1"])
    v = torch.lerp(g.square_(), v, a["beta2"])
    p = (s["master"] if c["master"] else s["p"]).to(f)
    up = (m / (1.0 - a["beta1"] ** c["step"]))
    up /= (v / (1.0 - a["beta2"] ** c["step"])).sqrt_() + a["eps"]
    p = p * s["factor64"][:, None] - a["lr"] * up
    out = {"p": p, "master": p} if c["master"] else {"p": p}
    if c["bits"] == 32:
        return {**out, "m": m, "v": v}
    return {**out, "m": None, "ms": m.abs().amax(1) / E4M3_MAX, "v": None,
            "vs": v.amax(1).sqrt() / E4M3_MAX}
