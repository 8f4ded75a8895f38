"""Products with 4-bit weights (moe_pack_weights_int4, moe_linear_int4 and the
4-bit layouts of moe_grouped_swiglu, moe_grouped_swiglu_fp8_rows and
moe_layer_forward) against plain fp64 forms, element by element within bounds
derived from the roundings each takes."""
import numpy as np
import pytest
import torch

import oracle
import synth
from _gpu_common import GAP_MIN, lib, need_gpu, np64, workspace
from _int4_common import bank, close, dequant64, dot_bound, fp8_rows, swiglu64, values64

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rows(gen, T, width, rows8):
    """(x, x_scale) on the GPU and their fp64 values."""
    x = torch.randn((T, width), generator=gen) * torch.exp2(torch.rand((T, 1), generator=gen) * 4)
    if rows8:
        q, s = fp8_rows(x)
        return q.cuda(), s.cuda(), values64(q, s)
    x = x.bfloat16()
    return x.cuda(), None, values64(x)


def _expected_packed(kind, q, s):
    """The packed bytes moe.h specifies, built on the CPU."""
    G, R, C2 = q.shape
    C, per = 2 * C2, 128 * s.shape[2] // (2 * C2)
    code = np.empty((G, R, C), dtype=np.uint32)
    code[:, :, 0::2], code[:, :, 1::2] = q & 15, q >> 4
    out = []
    for g in range(G):
        for b in range(R // 16):
            rows = [16 * b + r if kind == 1 else
                    (8 * b + r if r < 8 else R // 2 + 8 * b + r - 8) for r in range(16)]
            for ch in range(C // 128):
                words = np.zeros((2, 32, 4), dtype=np.uint32)
                for lane in range(32):
                    for i in range(8):
                        w = 0
                        for j in range(4):
                            row = rows[lane // 4 + 8 * (j % 2)]
                            col = 128 * ch + 32 * (i // 2) + 8 * (lane % 4) + 4 * (i % 2) + 2 * (j // 2)
                            w |= int(code[g, row, col]) << (4 * j)
                            w |= int(code[g, row, col + 1]) << (4 * j + 16)
                        words[i // 4, lane, i % 4] = w
                sc = [s[g, rows[r + 8 * hi], per * ch:per * ch + per] for r in range(8) for hi in (0, 1)]
                out.append(words.tobytes() + np.concatenate(sc).tobytes())
    return b"".join(out)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("kind,G,R,C", [(0, 2, 48, 256), (1, 3, 16, 128), (1, 1, 80, 384)])
def test_packed_bytes(kind, G, R, C, group):
    need_gpu()
    fgs = lib()
    q, s = bank(_gen(R + group), G, R, C, group)
    got = fgs.pack_int4(kind, q.cuda(), s.cuda())
    want = _expected_packed(kind, q.numpy(), s.view(torch.int16).numpy())
    assert got.cpu().numpy().tobytes() == want


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("rows8", [False, True])
@pytest.mark.parametrize("T,I,O,add", [
    (1, 128, 16, False), (1, 7168, 48, True), (1, 896, 4112, False), (2, 256, 272, True),
    (7, 384, 1040, False), (8, 2048, 160, True), (9, 128, 2448, False), (13, 3584, 64, True),
    (16, 1152, 96, False), (17, 640, 2432, True), (31, 7168, 32, False), (33, 512, 5008, True),
    (65, 1920, 112, False), (130, 256, 80, True), (3, 18432, 16, False), (40, 12288, 48, False),
    (2, 32768, 16, False), (128, 128, 144, False), (129, 128, 4112, True), (257, 384, 272, False),
    (300, 1152, 32, True), (18, 32768, 48, False),
])
def test_linear(T, I, O, add, rows8, group):
    need_gpu()
    fgs = lib()
    gen = _gen(T * 1000 + I + O)
    q, s = bank(gen, 1, O, I, group)
    x, xs, x64 = _rows(gen, T, I, rows8)
    W = fgs.pack_int4(fgs.MOE_PACK_PLAIN, q.cuda(), s.cuda())
    a = torch.randn((T, O), generator=gen).bfloat16().cuda() if add else None
    y = torch.full((T + 1, O), 7.0, dtype=torch.bfloat16, device="cuda")
    fgs.moe_linear_int4(T, I, O, group, x, xs, W, a, y)
    torch.cuda.synchronize()
    w = dequant64(q[0], s[0])
    ref, bound = x64 @ w.T, dot_bound(w, x64)
    if add:
        ref = ref + values64(a)
        bound = bound + 2.0 ** -23 * (np.abs(ref) + np.abs(values64(a)))
    close(y[:T], ref, bound)
    assert (y[T] == 7.0).all()  # nothing beyond row T


@pytest.mark.parametrize("rows8", [False, True])
def test_linear_output_may_be_the_addend(rows8):
    need_gpu()
    fgs = lib()
    gen = _gen(5)
    q, s = bank(gen, 1, 96, 512, 32)
    x, xs, x64 = _rows(gen, 11, 512, rows8)
    W = fgs.pack_int4(fgs.MOE_PACK_PLAIN, q.cuda(), s.cuda())
    a = torch.randn((11, 96), generator=gen).bfloat16().cuda()
    y = a.clone()
    fgs.moe_linear_int4(11, 512, 96, 32, x, xs, W, y, y)
    z = torch.empty_like(a)
    fgs.moe_linear_int4(11, 512, 96, 32, x, xs, W, a, z)
    assert torch.equal(y, z)


@pytest.mark.parametrize("rows8", [False, True])
@pytest.mark.parametrize("T", [3, 12, 40])
def test_linear_row_independence_and_nonfinite(T, rows8):
    """A NaN or an infinity in one row stays in that row's outputs, and the
    other rows' bits do not depend on it."""
    need_gpu()
    fgs = lib()
    gen = _gen(T)
    q, s = bank(gen, 1, 64, 384, 32)
    x, xs, _ = _rows(gen, T, 384, rows8)
    W = fgs.pack_int4(fgs.MOE_PACK_PLAIN, q.cuda(), s.cuda())
    y0 = torch.empty((T, 64), dtype=torch.bfloat16, device="cuda")
    fgs.moe_linear_int4(T, 384, 64, 32, x, xs, W, None, y0)
    bad = x.clone()
    if rows8:
        bad[1, 200] = 0x7F  # NaN code
    else:
        bad[1, 200] = float("nan")
    y1 = torch.empty_like(y0)
    fgs.moe_linear_int4(T, 384, 64, 32, bad, xs, W, None, y1)
    keep = [t for t in range(T) if t != 1]
    assert torch.isnan(y1[1]).all()
    assert torch.equal(y0[keep], y1[keep])


def test_linear_same_bits_every_run_and_on_a_side_stream():
    need_gpu()
    fgs = lib()
    gen = _gen(77)
    q, s = bank(gen, 1, 4096, 2048, 32)
    x, xs, _ = _rows(gen, 5, 2048, False)
    W = fgs.pack_int4(fgs.MOE_PACK_PLAIN, q.cuda(), s.cuda())
    outs = [torch.empty((5, 4096), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for i, y in enumerate(outs):
        fgs.moe_linear_int4(5, 2048, 4096, 32, x, xs, W, None, y,
                            stream=side if i % 2 else None)
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], y) for y in outs[1:])


# ---------------------------------------------------------------- experts
def _case(T, d, F, E, K, S, Fs, L, group, idx, rows8, seed, weights=True):
    """One moe_grouped_swiglu(_fp8_rows) call through moe_permute, and what it
    should give: (Y, Y_shared, permutation, refs and bounds)."""
    fgs = lib()
    gen = _gen(seed)
    de = L or d
    cfg = fgs.config(d_model=d, d_ff=F, E_routed=E, E_shared=S, d_ff_shared=Fs, K=K, d_latent=L,
                     weight_layout=3 if group == 32 else 4)
    banks = {"gu": bank(gen, E, 2 * F, de, group), "dn": bank(gen, E, de, F, group)}
    if S:
        banks["sgu"], banks["sdn"] = bank(gen, S, 2 * Fs, d, group), bank(gen, S, d, Fs, group)
    packed = {k: fgs.pack_int4(0 if "gu" in k else 1, q.cuda(), s.cuda())
              for k, (q, s) in banks.items()}
    xe, xes, xe64 = _rows(gen, T, de, rows8)
    if S and L:
        xs, xss, xs64 = _rows(gen, T, d, rows8)
    else:
        xs, xss, xs64 = xe, xes, xe64
    ws, nws = workspace(cfg, T)
    idx_t = torch.as_tensor(idx, dtype=torch.int32, device="cuda").contiguous()
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, perm, inv = i32(E), i32(E + 1), i32(T * K), i32(T * K)
    fgs.moe_permute(cfg, T, idx_t, counts, offsets, perm, inv, ws, nws)
    w = torch.rand((T, K), generator=gen) + 0.1 if weights else None
    wg = w.cuda() if weights else None
    Y = torch.full((T * K, de), 5.0, dtype=torch.bfloat16, device="cuda")
    Ysh = torch.full((max(S, 1) * T, d), 5.0, dtype=torch.bfloat16, device="cuda")
    args = (packed["gu"], packed["dn"])
    sh = (packed.get("sgu"), packed.get("sdn"))
    if rows8:
        fgs.moe_grouped_swiglu_fp8_rows(cfg, T, xe, xes, offsets, perm, wg, *args,
                                        xs if S else None, xss if S else None, *sh, Y,
                                        Ysh if S else None, ws, nws)
    else:
        fgs.moe_grouped_swiglu(cfg, T, xe, offsets, perm, wg, *args, xs if S else None, *sh, Y,
                               Ysh if S else None, ws, nws)
    torch.cuda.synchronize()
    off, pm = offsets.cpu().numpy(), perm.cpu().numpy()
    for e in range(E):
        if off[e + 1] == off[e]:
            continue
        pairs = pm[off[e]:off[e + 1]]
        y, b = swiglu64(xe64[pairs // K], dequant64(*[t[e] for t in banks["gu"]]),
                        dequant64(*[t[e] for t in banks["dn"]]))
        f = w.reshape(-1).numpy().astype(np.float64)[pairs][:, None] if weights else 1.0
        close(Y[off[e]:off[e + 1]], f * y, f * b * (1 + 2.0 ** -22))
    for i in range(S):
        y, b = swiglu64(xs64, dequant64(*[t[i] for t in banks["sgu"]]),
                        dequant64(*[t[i] for t in banks["sdn"]]))
        close(Ysh[i * T:(i + 1) * T], y, b)
    assert (Y[off[E]:] == 5.0).all()  # no write beyond the routed rows
    return Y, Ysh


def _random_idx(T, E, K, seed):
    g = np.random.default_rng(seed)
    return np.stack([g.choice(E, K, replace=False) for _ in range(T)])


@pytest.mark.parametrize("rows8", [False, True])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T,d,F,E,K,S,Fs,L", [
    (1, 256, 128, 16, 4, 1, 128, 0),      # one token
    (1, 1024, 384, 5, 1, 0, 0, 0),        # no shared expert, K = 1
    (5, 384, 256, 12, 3, 2, 384, 0),
    (9, 256, 128, 4, 4, 1, 256, 0),       # K = E: every expert has every token
    (40, 512, 128, 48, 6, 1, 128, 256),   # latent form, most experts with a few rows
    (70, 256, 384, 8, 2, 1, 128, 0),      # tiles of rows that end inside an expert
    (3, 7168, 128, 6, 2, 1, 128, 0),      # the widest rows
    (300, 384, 256, 5, 2, 2, 128, 0),     # several tiles of tokens an expert
    (200, 256, 128, 6, 3, 1, 384, 512),   # and the latent form
])
def test_experts(T, d, F, E, K, S, Fs, L, group, rows8):
    need_gpu()
    _case(T, d, F, E, K, S, Fs, L, group, _random_idx(T, E, K, T + E), rows8, T + d)


@pytest.mark.parametrize("rows8", [False, True])
def test_experts_all_tokens_on_one_expert(rows8):
    need_gpu()
    T = 45
    _case(T, 256, 128, 32, 1, 0, 0, 0, 32, np.full((T, 1), 31), rows8, 3)


@pytest.mark.parametrize("rows8", [False, True])
def test_experts_of_every_size(rows8):
    """Experts with 0, 1, 2, ... rows in one call, over every kernel's range."""
    need_gpu()
    sizes = [0, 1, 2, 7, 8, 9, 15, 16, 17, 18, 31, 32, 33, 63, 0, 64, 65, 127, 128, 129, 200]
    idx = np.concatenate([np.full(n, e) for e, n in enumerate(sizes)])
    np.random.default_rng(3).shuffle(idx)
    _case(len(idx), 256, 128, len(sizes), 1, 0, 0, 0, 32, idx[:, None], rows8, 11)


def test_experts_named_twice_by_a_token():
    """moe_grouped_swiglu takes any grouping: an expert may have more rows
    than there are tokens."""
    need_gpu()
    for T in (6, 14, 40):
        idx = np.stack([np.full(T, 3), np.full(T, 3), np.arange(T) % 5], axis=1)
        _case(T, 256, 128, 8, 3, 1, 128, 0, 32, idx, False, 12)


def test_experts_without_weights_and_with_rejected_pairs():
    """Pairs with an expert index outside [0, E) have no slot: the rows that
    remain are right and the ones behind them are left alone."""
    need_gpu()
    idx = _random_idx(20, 16, 4, 9)
    idx[3, 1], idx[19, 0] = -1, 16
    _case(20, 256, 128, 16, 4, 1, 128, 0, 32, idx, False, 4, weights=False)
    # every pair rejected: no routed row at all
    _case(4, 256, 128, 8, 2, 1, 128, 0, 32, np.full((4, 2), -1), False, 6)


def test_experts_same_bits_every_run():
    need_gpu()
    idx = _random_idx(33, 24, 3, 1)
    a = _case(33, 512, 256, 24, 3, 1, 256, 0, 32, idx, False, 8)
    b = _case(33, 512, 256, 24, 3, 1, 256, 0, 32, idx, False, 8)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_experts_banks_beyond_4_gib():
    """The last experts of a bank of more than 2^32 bytes."""
    need_gpu()
    fgs = lib()
    E, d, F, T, K = 300, 7168, 2048, 2, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    banks = {}
    for k, rows, cols in (("gu", 2 * F, d), ("dn", d, F)):
        q = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = (torch.rand((E, rows, cols // 32), generator=g, device="cuda") * 0.01).bfloat16()
        banks[k] = (q, s, fgs.pack_int4(0 if k == "gu" else 1, q, s))
    assert banks["gu"][2].numel() > 1 << 32
    cfg = fgs.config(d_model=d, d_ff=F, E_routed=E, K=K, weight_layout=3)
    ws, nws = workspace(cfg, T)
    x = torch.randn((T, d), generator=g, device="cuda").bfloat16()
    perm = torch.tensor([1, 2, 0, 3], dtype=torch.int32, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E - 1:] = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    Y = torch.empty((T * K, d), dtype=torch.bfloat16, device="cuda")
    fgs.moe_grouped_swiglu(cfg, T, x, off, perm, None, banks["gu"][2], banks["dn"][2], None, None,
                           None, Y, None, ws, nws)
    for e, rows in ((E - 2, [0, 1]), (E - 1, [0, 1])):
        y, b = swiglu64(values64(x)[rows], dequant64(*[t[e] for t in banks["gu"][:2]]),
                        dequant64(*[t[e] for t in banks["dn"][:2]]))
        lo = 0 if e == E - 2 else 2
        close(Y[lo:lo + 2], y, b)


@pytest.mark.parametrize("L", [0, 256])
@pytest.mark.parametrize("group", [32, 128])
def test_layer_forward(group, L):
    """moe_layer_forward in a 4-bit layout against the oracle layer on the
    dequantised weights."""
    need_gpu()
    fgs = lib()
    shape = synth.custom(name="int4_layer", T=37, d_model=512, E_routed=24, K=4, E_shared=1,
                         d_ff=128, d_ff_shared=256, n_group=4, topk_group=2, d_latent=L)
    T, d, E, S = shape.T, shape.d_model, shape.E_routed, 1
    de = L or d
    gen = _gen(group + L)
    x = synth.activations(shape, "cuda")
    W_r, bias = synth.router_params(shape, "cuda")
    dims = {"W_gate_up": (E, 256, de), "W_down": (E, de, 128), "Ws_gate_up": (S, 512, d),
            "Ws_down": (S, d, 256)}
    raw, packed = {}, {}
    for k, (n, r, c) in dims.items():
        q, s = bank(gen, n, r, c, group)
        s = s * 0.25
        raw[k] = torch.from_numpy(np.stack([dequant64(q[i], s[i]) for i in range(n)]))
        packed[k] = fgs.pack_int4(0 if "gate_up" in k else 1, q.cuda(), s.cuda())
    lat = {}
    if L:
        lat["W_lat_down"], lat["W_lat_up"] = synth.latent_projections(shape, "cuda")
    lp = fgs.pack_layer_weights(dict(lat)) if L else {}
    cfg = fgs.config(shape, weight_layout=3 if group == 32 else 4)
    ws, nws = workspace(cfg, T)
    y = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    idx = torch.empty((T, 4), dtype=torch.int32, device="cuda")
    fgs.moe_layer_forward(cfg, T, x, W_r, bias, packed["W_gate_up"], packed["W_down"],
                          packed["Ws_gate_up"], packed["Ws_down"], lp.get("W_lat_down"),
                          lp.get("W_lat_up"), y, idx, None, None, ws, nws)
    assert fgs.moe_get_device_status(ws) == 0
    kw = dict(W_lat_down64=np64(lat["W_lat_down"]), W_lat_up64=np64(lat["W_lat_up"])) if L else {}
    ref = oracle.moe_layer_tokens(np64(x), np64(W_r), bias.cpu().numpy(), raw["W_gate_up"],
                                  raw["W_down"], raw["Ws_gate_up"], raw["Ws_down"], 4, 4, 2,
                                  to_f64=lambda t: t.numpy() if torch.is_tensor(t) else t, **kw)
    same = (np.sort(idx.cpu().numpy(), 1) == np.sort(ref["idx"], 1)).all(1)
    assert same[ref["gap"] > GAP_MIN].all()
    # bf16 roundings of x's projection, H, Y, the routed sum and y: 2^-8 each
    # of terms that sum with at most a factor of a few to max |y|
    err = np.abs(np64(y)[same] - ref["y"][same]).max() / np.abs(ref["y"][same]).max()
    assert err <= 1e-2


def test_host_forward_takes_the_layout():
    need_gpu()
    fgs = lib()
    shape = synth.custom(name="int4_host", T=8, d_model=256, E_routed=8, K=2, E_shared=1, d_ff=128,
                         d_ff_shared=128)
    gen = _gen(2)
    p = {k: fgs.pack_int4(kind, *[t.cuda() for t in bank(gen, *dims, 32)])
         for k, kind, dims in (("gu", 0, (8, 256, 256)), ("dn", 1, (8, 256, 128)),
                               ("sgu", 0, (1, 256, 256)), ("sdn", 1, (1, 256, 128)))}
    x = synth.activations(shape, "cuda")
    W_r, bias = synth.router_params(shape, "cuda")
    cfg = fgs.config(shape, weight_layout=3)
    ws, nws = workspace(cfg, 8)
    y = torch.empty_like(x)
    fgs.moe_layer_forward(cfg, 8, x, W_r, bias, p["gu"], p["dn"], p["sgu"], p["sdn"], None, None, y,
                          None, None, None, ws, nws)
    xh, yh = x.cpu().pin_memory(), torch.empty(x.shape, dtype=x.dtype).pin_memory()
    fgs.moe_layer_forward_host(cfg, 8, xh, W_r, bias, p["gu"], p["dn"], p["sgu"], p["sdn"], None,
                               None, yh, ws, nws)
    torch.cuda.synchronize()
    fgs.moe_layer_forward_host_release(ws)
    assert torch.equal(y.cpu(), yh)


@pytest.mark.parametrize("rows8", [False, True])
@pytest.mark.parametrize("T,L,S,group", [(1, 0, 1, 32), (5, 0, 2, 128), (50, 256, 2, 32),
                                         (60, 0, 1, 128), (3, 256, 0, 32)])
def test_decode_block(T, L, S, group, rows8):
    """The norm, router, experts and combine of run_decode together against
    its plain fp32 form."""
    need_gpu()
    lib()
    from fine_grained_sparse_gb300.run_decode import Block, plain_block
    shape = synth.custom(name="block", T=T, d_model=512, E_routed=16, K=4, E_shared=S, d_ff=256,
                         d_ff_shared=128 if S else 0, d_latent=L)
    b = Block(shape, T, group, rows8, keep=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    attn, res = (torch.randn((T, 512), generator=g, device="cuda").bfloat16() for _ in range(2))
    h, y = b(attn, res)
    ph, py = plain_block(b, attn, res)
    # h: one bf16 rounding, 2^-8.  y, as norms over all elements: independent
    # roundings of x (bf16, or E4M3's 2^-4), the latent rows, H, Y, the routed
    # sum and y; a unit of 2^-p is an error of at most 2^-p / sqrt(3) of an
    # element in the mean, which SwiGLU's two factors at most double
    assert float((h.float() - ph).norm() / ph.norm()) <= 2.0 ** -8
    u = np.sqrt((2 * (2.0 ** -4 if rows8 else 2.0 ** -8)) ** 2 + 6 * (2.0 ** -8) ** 2) / np.sqrt(3)
    assert float((y.float() - py).norm() / py.norm()) <= u


@pytest.mark.parametrize("rows8", [False, True])
def test_calls_in_a_captured_graph(rows8):
    """The calls enqueue nothing but kernels: they can be captured, and every
    replay reads what its inputs hold then."""
    need_gpu()
    fgs = lib()
    gen = _gen(21)
    shape = dict(T=50, d=256, F=128, E=6, K=2)
    T, d, F, E, K = shape.values()
    cfg = fgs.config(d_model=d, d_ff=F, E_routed=E, K=K, weight_layout=3)
    gu, dn = (fgs.pack_int4(kind, *[t.cuda() for t in bank(gen, E, r, c, 32)])
              for kind, r, c in ((0, 2 * F, d), (1, d, F)))
    W = fgs.pack_int4(1, *[t.cuda() for t in bank(gen, 1, 96, d, 32)])
    x, xs, _ = _rows(gen, T, d, rows8)
    ws, nws = workspace(cfg, T)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, perm, inv = i32(E), i32(E + 1), i32(T * K), i32(T * K)
    idx = torch.as_tensor(_random_idx(T, E, K, 5), dtype=torch.int32, device="cuda")
    Y, y = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((T * K, d), (T, 96)))

    def step():
        fgs.moe_permute(cfg, T, idx, counts, offsets, perm, inv, ws, nws)
        if rows8:
            fgs.moe_grouped_swiglu_fp8_rows(cfg, T, x, xs, offsets, perm, None, gu, dn, None, None,
                                            None, None, Y, None, ws, nws)
        else:
            fgs.moe_grouped_swiglu(cfg, T, x, offsets, perm, None, gu, dn, None, None, None, Y,
                                   None, ws, nws)
        fgs.moe_linear_int4(T, d, 96, 32, x, xs, W, None, y)

    step()
    torch.cuda.synchronize()
    first = (Y.clone(), y.clone())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    Y.zero_(), y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, first[0]) and torch.equal(y, first[1])
    new = torch.as_tensor(_random_idx(T, E, K, 6), dtype=torch.int32, device="cuda")
    idx.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    again = Y.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(Y, again) and not torch.equal(Y, first[0])
