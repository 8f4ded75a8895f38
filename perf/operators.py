"""The measured cases of the 4-bit decode operators: the residual sum with its
RMS norm (``moe_add_rmsnorm``), the linear map with 4-bit weights
(``moe_linear_int4``) and the SwiGLU experts with 4-bit weights
(``moe_grouped_swiglu`` / ``moe_grouped_swiglu_fp8_rows``).

With ``own`` false ``run`` computes an operator in elementary torch operations
in fp32, rounded once at the end; with ``own`` true it makes the library's
calls.  A 4-bit weight is (code - 8) * scale, two codes to a byte (the even
column in the low half), one bf16 scale for ``group`` columns of a row.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
ROW_GROUP = 128  # columns of a row that share one scale of the 8-bit form
EPS = 1e-6


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of one sequence, before the layer: latency
        {"name": "norm T1 d7168 fp8", "op": "norm", "T": 1, "d": 7168, "dtype": "bf16",
         "residual": True, "y": True, "fp8": True},
        # a batch of fp32 rows of a width that no power of two divides
        {"name": "norm T333 d1000 f32", "op": "norm", "T": 333, "d": 1000, "dtype": "f32",
         "residual": True, "y": True, "fp8": False},
        # the layer's prefill batch: bandwidth
        {"name": "norm T8192 d7168 fp8", "op": "norm", "T": 8192, "d": 7168, "dtype": "bf16",
         "residual": True, "y": True, "fp8": True},
        # one token through a latent down-projection
        {"name": "linear T1 7168-3584 g32", "op": "linear", "T": 1, "I": 7168, "O": 3584,
         "group": 32, "rows8": False, "add": False},
        # an odd batch through the up-projection, added to a running sum, rows in 8 bits
        {"name": "linear T13 3584-7168 g128 fp8", "op": "linear", "T": 13, "I": 3584, "O": 7168,
         "group": 128, "rows8": True, "add": True},
        # a decode batch through a wide projection
        {"name": "linear T64 7168-18432 g32", "op": "linear", "T": 64, "I": 7168, "O": 18432,
         "group": 32, "rows8": False, "add": False},
        # one token through its top-8 experts and the shared one
        {"name": "experts T1 of 384 g32", "op": "experts", "T": 1, "d": 7168, "F": 2048, "E": 384,
         "U": 8, "K": 8, "S": 1, "Fs": 2048, "dl": 0, "group": 32, "rows8": False},
        # a few sequences decoded together, rows in 8 bits from the norm
        {"name": "experts T8 of 384 g32 fp8", "op": "experts", "T": 8, "d": 7168, "F": 2048,
         "E": 384, "U": 56, "K": 8, "S": 1, "Fs": 2048, "dl": 0, "group": 32, "rows8": True},
        # the layer's decode batch: nearly every expert is read for a few rows
        {"name": "experts T128 of 384 g32", "op": "experts", "T": 128, "d": 7168, "F": 2048,
         "E": 384, "U": 357, "K": 8, "S": 1, "Fs": 2048, "dl": 0, "group": 32, "rows8": False},
        # the latent form: routed experts of another width than the shared ones
        {"name": "experts T24 of 896 latent g32", "op": "experts", "T": 24, "d": 7168, "F": 3072,
         "E": 896, "U": 300, "K": 16, "S": 2, "Fs": 3072, "dl": 3584, "group": 32,
         "rows8": False},
        # small experts, a ragged batch with popular experts, groups of 128
        {"name": "experts T301 of 64 g128", "op": "experts", "T": 301, "d": 1920, "F": 640,
         "E": 64, "U": 61, "K": 6, "S": 1, "Fs": 1280, "dl": 0, "group": 128, "rows8": False},
        # a larger decode batch: several rows for every expert, rows in 8 bits
        {"name": "experts T512 of 384 g128 fp8", "op": "experts", "T": 512, "d": 7168, "F": 2048,
         "E": 384, "U": 384, "K": 8, "S": 1, "Fs": 2048, "dl": 0, "group": 128, "rows8": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "experts", "experts", "experts"])
    if op == "norm":
        fp8 = rng.random() < 0.6
        d = 128 * _log(rng, 1, 64) if fp8 else _log(rng, 64, 8192)
        T = max(1, min(_log(rng, 1, 8192), 8192 * 7168 // d))
        return {"op": op, "T": T, "d": d, "dtype": "bf16" if rng.random() < 0.75 else "f32",
                "residual": rng.random() < 0.8, "y": (not fp8) or rng.random() < 0.7, "fp8": fp8}
    group = rng.choice([32, 32, 128])
    rows8 = rng.random() < 0.4
    if op == "linear":
        return {"op": op, "T": _log(rng, 1, 64), "I": 128 * _log(rng, 2, 56),
                "O": 16 * _log(rng, 16, 1152), "group": group, "rows8": rows8,
                "add": rng.random() < 0.4}
    E = rng.choice([16, 48, 64, 128, 256, 384])
    K = rng.choice([1, 2, 4, 6, 8])
    T = _log(rng, 1, 512)
    d = 128 * _log(rng, 4, 56)
    F = 128 * _log(rng, 1, 16)
    U = min(E, T * K) if T * K <= K else rng.randint(min(E, K), min(E, T * K))
    S = rng.choice([0, 1, 1, 2])
    return {"op": op, "T": T, "d": d, "F": F, "E": E, "U": U, "K": K, "S": S,
            "Fs": 128 * _log(rng, 1, 16), "dl": 128 * rng.randint(2, max(2, d // 256))
            if rng.random() < 0.25 else 0, "group": group, "rows8": rows8}


def work(case):
    c = case
    T = c["T"]
    if c["op"] == "norm":
        d, b = c["d"], 2 if c["dtype"] == "bf16" else 4
        tensors = 1 + 2 * c["residual"] + c["y"]  # a, (r, h), y
        n = T * d * b * tensors + d * b + (T * d + 4 * T * (d // ROW_GROUP)) * c["fp8"]
        return {"bytes": n, "flops": 6 * T * d}
    per_weight = 0.5 + 2.0 / c["group"]

    def rows(n, width):
        return n * (width + 4 * (width // ROW_GROUP)) if c["rows8"] else 2 * n * width

    if c["op"] == "linear":
        I, O = c["I"], c["O"]
        return {"bytes": int(I * O * per_weight + rows(T, I) + 2 * T * O * (1 + c["add"])),
                "flops": 2 * T * I * O}
    de = c["dl"] or c["d"]
    routed, shared = 3 * c["F"] * de, 3 * c["Fs"] * c["d"]
    n = (c["U"] * routed + c["S"] * shared) * per_weight
    n += rows(T, de) + (rows(T, c["d"]) if c["S"] and c["dl"] else 0)
    n += 2 * T * c["K"] * de + 2 * c["S"] * T * c["d"] + 8 * T * c["K"] + 4 * (c["E"] + 1)
    return {"bytes": int(n), "flops": 2 * T * (c["K"] * routed + c["S"] * shared)}


# --------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _codes(g, *shape):
    """4-bit codes, two to a byte: all byte values, so all code pairs."""
    return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)


def _scales(g, *shape):
    """Scales that make weights of about N(0, 0.02)-sized values."""
    return (torch.rand(shape, generator=g, device="cuda") + 0.5).mul_(0.02 / 4.6).bfloat16()


def _bank(g, groups, rows, cols, group):
    return {"q": _codes(g, groups, rows, cols // 2), "s": _scales(g, groups, rows, cols // group)}


def _rows(g, T, width, rows8):
    """Normalised activations, some columns larger than the others as a norm's
    weights make them; in bf16, or in E4M3 with a scale per 128 columns."""
    x = torch.randn((T, width), generator=g, device="cuda")
    x *= torch.rand((width,), generator=g, device="cuda") + 0.5
    if not rows8:
        return {"x": x.bfloat16(), "xs": None}
    m = x.view(T, width // ROW_GROUP, ROW_GROUP)
    xs = (m.abs().amax(-1) / E4M3_MAX).clamp_min(1e-30)
    return {"x": (m / xs[..., None]).to(torch.float8_e4m3fn).view(T, width), "xs": xs}


def _routing(g, case):
    """topk_idx [T, K] that reaches exactly U experts: the first tokens walk
    through a random subset of the experts, the others draw theirs from it
    with popularities that differ by a factor of ten; and random weights."""
    T, K, E, U = case["T"], case["K"], case["E"], case["U"]
    subset = torch.randperm(E, generator=g, device="cuda")[:U]
    need = -(-U // K)
    popular = torch.rand((U,), generator=g, device="cuda") * math.log(10.0)
    noise = torch.rand((T, U), generator=g, device="cuda").clamp_min_(1e-9)
    pick = (popular - torch.log(-torch.log(noise).clamp_min_(1e-9))).topk(K, dim=1).indices
    walk = torch.arange(need * K, device="cuda").view(need, K) % U
    pick[:need] = walk
    pick = pick[torch.randperm(T, generator=g, device="cuda")]
    w = torch.rand((T, K), generator=g, device="cuda") + 0.05
    w = 2.827 * w / w.sum(1, keepdim=True)
    return subset[pick].to(torch.int32), w


def prepare(case, seed):
    g = _generator(seed)
    c, st = case, {"case": dict(case)}
    T = c["T"]
    if c["op"] == "norm":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        st["a"] = torch.randn((T, c["d"]), generator=g, device="cuda").to(dt)
        if c["residual"]:
            st["r"] = (3.0 * torch.randn((T, c["d"]), generator=g, device="cuda")).to(dt)
        st["w"] = (1.0 + 0.2 * torch.randn((c["d"],), generator=g, device="cuda")).to(dt)
        if own:
            import fine_grained_sparse_gb300 as fgs
            st["fgs"] = fgs
            st["dt"] = fgs.MOE_BF16 if c["dtype"] == "bf16" else fgs.MOE_F32
            st["h"] = torch.empty_like(st["a"]) if c["residual"] else None
            st["y"] = torch.empty_like(st["a"]) if c["y"] else None
            if c["fp8"]:
                st["y8"] = torch.empty((T, c["d"]), dtype=torch.float8_e4m3fn, device="cuda")
                st["ys"] = torch.empty((T, c["d"] // ROW_GROUP), device="cuda")
        return st
    if c["op"] == "linear":
        st.update(_rows(g, T, c["I"], c["rows8"]))
        W = _bank(g, 1, c["O"], c["I"], c["group"])
        if c["add"]:
            st["add"] = torch.randn((T, c["O"]), generator=g, device="cuda").bfloat16()
        if own:
            import fine_grained_sparse_gb300 as fgs
            st["fgs"] = fgs
            st["W"] = fgs.pack_int4(fgs.MOE_PACK_PLAIN, W["q"], W["s"])
            st["y"] = torch.empty((T, c["O"]), dtype=torch.bfloat16, device="cuda")
        else:
            st["W"] = W
        return st
    d, de, E, S = c["d"], c["dl"] or c["d"], c["E"], c["S"]
    st.update(_rows(g, T, de, c["rows8"]))
    if S and c["dl"]:
        both = _rows(g, T, d, c["rows8"])
        st["xsh"], st["xshs"] = both["x"], both["xs"]
    elif S:
        st["xsh"], st["xshs"] = st["x"], st["xs"]
    idx, st["topk_w"] = _routing(g, c)
    flat = idx.reshape(-1)
    st["perm"] = torch.sort(flat, stable=True).indices.to(torch.int32)
    counts = torch.bincount(flat, minlength=E)
    st["offsets"] = torch.zeros((E + 1,), dtype=torch.int32, device="cuda")
    st["offsets"][1:] = counts.cumsum(0)
    banks = {"W_gate_up": (E, 2 * c["F"], de), "W_down": (E, de, c["F"])}
    if S:
        banks.update(Ws_gate_up=(S, 2 * c["Fs"], d), Ws_down=(S, d, c["Fs"]))
    if own:
        import fine_grained_sparse_gb300 as fgs
        st["fgs"] = fgs
    for name, (n, rows, cols) in banks.items():
        bank = _bank(g, n, rows, cols, c["group"])
        if own:
            kind = fgs.MOE_PACK_GATE_UP if "gate_up" in name else fgs.MOE_PACK_PLAIN
            bank = fgs.pack_int4(kind, bank["q"], bank["s"])
        st[name] = bank
    if own:
        layout = {32: fgs.MOE_WEIGHTS_PACKED_INT4_G32, 128: fgs.MOE_WEIGHTS_PACKED_INT4_G128}
        st["cfg"] = fgs.config(d_model=d, d_ff=c["F"], E_routed=E, E_shared=S,
                               d_ff_shared=c["Fs"] if S else 0, K=c["K"], d_latent=c["dl"],
                               weight_layout=layout[c["group"]])
        st["nws"] = fgs.moe_workspace_size(st["cfg"], T)
        st["ws"] = torch.zeros(st["nws"], dtype=torch.uint8, device="cuda")
        st["Y"] = torch.empty((T * c["K"], de), dtype=torch.bfloat16, device="cuda")
        if S:
            st["Ysh"] = torch.empty((S, T, d), dtype=torch.bfloat16, device="cuda")
    else:
        # the plan of a plain program: which experts have rows, and which slots
        off = st["offsets"].tolist()
        st["present"] = [(e, off[e], off[e + 1]) for e in range(E) if off[e + 1] > off[e]]
    return st


# -------------------------------------------------------------- the two forms
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "experts": _own_experts}[op](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "experts": _plain_experts}[op](state)


def _own_norm(s):
    c = s["case"]
    s["fgs"].moe_add_rmsnorm(s["dt"], c["T"], c["d"], s["a"], s.get("r"), s["w"], EPS, s["h"],
                             s["y"], s.get("y8"), s.get("ys"))
    return {k: s.get(k) for k in ("h", "y", "y8", "ys") if s.get(k) is not None}


def _own_linear(s):
    c = s["case"]
    s["fgs"].moe_linear_int4(c["T"], c["I"], c["O"], c["group"], s["x"], s["xs"], s["W"],
                             s.get("add"), s["y"])
    return {"y": s["y"]}


def _own_experts(s):
    c, fgs = s["case"], s["fgs"]
    banks = (s["W_gate_up"], s["W_down"])
    shared = (s.get("Ws_gate_up"), s.get("Ws_down"))
    if c["rows8"]:
        fgs.moe_grouped_swiglu_fp8_rows(s["cfg"], c["T"], s["x"], s["xs"], s["offsets"], s["perm"],
                                        s["topk_w"], *banks, s.get("xsh"), s.get("xshs"), *shared,
                                        s["Y"], s.get("Ysh"), s["ws"], s["nws"])
    else:
        fgs.moe_grouped_swiglu(s["cfg"], c["T"], s["x"], s["offsets"], s["perm"], s["topk_w"],
                               *banks, s.get("xsh"), *shared, s["Y"], s.get("Ysh"), s["ws"],
                               s["nws"])
    return {"Y": s["Y"], "Y_shared": s["Ysh"]} if c["S"] else {"Y": s["Y"]}


def _plain_norm(s):
    c = s["case"]
    out = {}
    v = s["a"].float()
    if c["residual"]:
        v = v + s["r"].float()
        out["h"] = v.to(s["a"].dtype)
    v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["w"].float()
    if c["y"]:
        out["y"] = v.to(s["a"].dtype)
    if c["fp8"]:
        m = v.view(c["T"], -1, ROW_GROUP)
        ys = m.abs().amax(-1) / E4M3_MAX
        q = torch.where(ys[..., None] > 0, m / ys[..., None], torch.zeros_like(m))
        out["y8"] = q.to(torch.float8_e4m3fn).view(c["T"], c["d"])
        out["ys"] = ys
    return out


def _weights(q, s):
    """fp32 weights [rows, cols] of codes [rows, cols / 2] and their scales."""
    v = torch.stack((q & 15, q >> 4), -1).view(q.shape[0], s.shape[1], -1).float()
    return ((v - 8.0) * s.float()[..., None]).view(q.shape[0], -1)


def _values(x, xs):
    x = x.float()
    if xs is None:
        return x
    return (x.view(x.shape[0], -1, ROW_GROUP) * xs[..., None]).view(x.shape)


def _plain_linear(s):
    y = _values(s["x"], s["xs"]) @ _weights(s["W"]["q"][0], s["W"]["s"][0]).t()
    if s["case"]["add"]:
        y = y + s["add"].float()
    return {"y": y.bfloat16()}


def _swiglu(u, gate_up, down):
    g, v = (u @ gate_up.t()).chunk(2, dim=1)
    return (g / (1.0 + torch.exp(-g)) * v) @ down.t()


def _plain_experts(s):
    c = s["case"]
    x = _values(s["x"], s["xs"])
    perm = s["perm"].long()
    wt = s["topk_w"].reshape(-1)[perm]
    Y = torch.empty((c["T"] * c["K"], x.shape[1]), dtype=torch.bfloat16, device="cuda")
    gu, dn = s["W_gate_up"], s["W_down"]
    for e, a, b in s["present"]:  # one expert's weights in fp32 at a time
        y = _swiglu(x[perm[a:b] // c["K"]], _weights(gu["q"][e], gu["s"][e]),
                    _weights(dn["q"][e], dn["s"][e]))
        Y[a:b] = (y * wt[a:b, None]).bfloat16()
    if not c["S"]:
        return {"Y": Y}
    xsh, gu, dn = _values(s["xsh"], s["xshs"]), s["Ws_gate_up"], s["Ws_down"]
    Ysh = torch.stack([_swiglu(xsh, _weights(gu["q"][i], gu["s"][i]),
                               _weights(dn["q"][i], dn["s"][i])).bfloat16()
                       for i in range(c["S"])])
    return {"Y": Y, "Y_shared": Ysh}


# -------------------------------------------------------------- in 64 bits
def _dequant64(bank, i):
    """Expert i's weights in fp64, column by column pair from the bytes."""
    q, s = bank["q"][i], bank["s"][i].double()
    w = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device="cuda")
    w[:, 0::2] = (q % 16).double() - 8.0
    w[:, 1::2] = torch.div(q, 16, rounding_mode="floor").double() - 8.0
    return w * s.repeat_interleave(w.shape[1] // s.shape[1], dim=1)


def _rows64(x, xs):
    v = x.float().double()
    return v if xs is None else v * xs.double().repeat_interleave(ROW_GROUP, dim=1)


def exact(case, seed):
    """What ``run`` returns from the definitions in fp64 (None for the 8-bit
    codes' place: their scale's last bit decides some of them)."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, out = case, {}
    if c["op"] == "norm":
        h = s["a"].double() + (s["r"].double() if c["residual"] else 0.0)
        if c["residual"]:
            out["h"] = h
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / c["d"] + EPS) * s["w"].double()
        if c["y"]:
            out["y"] = y
        if c["fp8"]:
            out["y8"] = None
            out["ys"] = y.abs().unflatten(1, (-1, ROW_GROUP)).max(2).values / E4M3_MAX
        return out
    if c["op"] == "linear":
        y = torch.matmul(_rows64(s["x"], s["xs"]), _dequant64(s["W"], 0).T)
        return {"y": y + s["add"].double() if c["add"] else y}

    def expert(u, gu, dn, i, F):
        z = torch.matmul(u, _dequant64(gu, i).T)
        return torch.matmul(z[:, :F] * torch.sigmoid(z[:, :F]) * z[:, F:], _dequant64(dn, i).T)

    x = _rows64(s["x"], s["xs"])
    Y = torch.empty((c["T"] * c["K"], x.shape[1]), dtype=torch.float64, device="cuda")
    for e, a, b in s["present"]:
        slots = s["perm"][a:b].long()
        y = expert(x[torch.div(slots, c["K"], rounding_mode="floor")], s["W_gate_up"],
                   s["W_down"], e, c["F"])
        Y[a:b] = y * s["topk_w"].view(-1)[slots].double()[:, None]
    out["Y"] = Y
    if c["S"]:
        xs = _rows64(s["xsh"], s["xshs"])
        out["Y_shared"] = torch.stack([expert(xs, s["Ws_gate_up"], s["Ws_down"], i, c["Fs"])
                                       for i in range(c["S"])])
    return out
