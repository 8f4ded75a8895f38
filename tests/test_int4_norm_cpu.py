"""Refusals of the 4-bit products and of the RMS norm, which come before any
CUDA call, and the sizes of packed 4-bit banks."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def fgs():
    import __graft_entry__
    __graft_entry__.build()
    import fine_grained_sparse_gb300 as m
    return m


P = [0x100000 * (i + 1) for i in range(16)]  # aligned addresses, never dereferenced


def test_packed_int4_bytes(fgs):
    # records of 16 x 128 codes and 16 x (128 / group) bf16 scales
    assert fgs.moe_packed_int4_bytes(384, 4096, 7168, 32) == 384 * 256 * 56 * (1024 + 128)
    assert fgs.moe_packed_int4_bytes(1, 16, 128, 128) == 1024 + 32
    for bad in [(0, 16, 128, 32), (1, 24, 128, 32), (1, 16, 64, 32), (1, 16, 192, 32),
                (1, 16, 128, 64), (1, 0, 128, 32)]:
        assert fgs.moe_packed_int4_bytes(*bad) == -1


@pytest.mark.parametrize("args,status", [
    ((5, 1, 16, 128, 32, P[0], P[1], P[2]), 1),            # kind
    ((1, 0, 16, 128, 32, P[0], P[1], P[2]), 1),            # groups
    ((1, 1, 24, 128, 32, P[0], P[1], P[2]), 2),            # rows % 16
    ((1, 1, 16, 192, 32, P[0], P[1], P[2]), 2),            # cols % 128
    ((1, 1, 16, 128, 64, P[0], P[1], P[2]), 2),            # group size
    ((1, 1, 16, 128, 32, None, P[1], P[2]), 1),
    ((1, 1, 16, 128, 32, P[0] + 8, P[1], P[2]), 3),
    ((1, 1, 16, 128, 32, P[0], P[1] + 1, P[2]), 3),
    ((1, 1, 16, 128, 32, P[0], P[1], P[0]), 1),            # overlap
    ((1, 1, 16, 128, 32, P[0], P[1], P[1] - 16), 1),       # overlap with the scales
])
def test_pack_refusals(fgs, args, status):
    assert fgs.lib.moe_pack_weights_int4(*args, None) == status


@pytest.mark.parametrize("kw,status", [
    ({}, 0),
    ({"d_ff": 2048 - 64}, 2),
    ({"d_ff_shared": 192}, 2),
    ({"d_model": 7168 + 64}, 2),
    ({"d_latent": 3584 - 64}, 2),
    ({"d_latent": 3584}, 0),
    ({"dtype": 0}, 2),
    ({"d_model": 32896}, 2),
    ({"weight_layout": 5}, 1),
])
@pytest.mark.parametrize("layout", [3, 4])
def test_validate_config(fgs, layout, kw, status):
    base = dict(d_model=7168, d_ff=2048, E_routed=384, E_shared=1, d_ff_shared=2048, K=8,
                dtype=fgs.MOE_BF16, weight_layout=layout)
    base.update(kw)
    assert fgs.moe_validate_config(fgs.config(**base), 128) == status


@pytest.mark.parametrize("args,status", [
    ((0, 256, 64, 32, P[0], None, P[1], None, P[2]), 1),       # T
    ((1, 200, 64, 32, P[0], None, P[1], None, P[2]), 2),
    ((1, 256, 72, 32, P[0], None, P[1], None, P[2]), 2),
    ((1, 32896, 64, 32, P[0], None, P[1], None, P[2]), 2),     # too wide
    ((1, 256, 64, 16, P[0], None, P[1], None, P[2]), 2),
    ((1, 256, 64, 32, None, None, P[1], None, P[2]), 1),
    ((1, 256, 64, 32, P[0], None, P[1], None, None), 1),
    ((1, 256, 64, 32, P[0] + 2, None, P[1], None, P[2]), 3),
    ((1, 256, 64, 32, P[0], P[3] + 4, P[1], None, P[2]), 3),
    ((1, 256, 64, 32, P[0], None, P[1], P[4] + 2, P[2]), 3),
])
def test_linear_refusals(fgs, args, status):
    assert fgs.lib.moe_linear_int4(*args, None) == status


def _swiglu(fgs, layout, **over):
    cfg = fgs.config(d_model=256, d_ff=128, E_routed=8, K=2, E_shared=1, d_ff_shared=128,
                     weight_layout=layout)
    a = dict(x=P[0], xs=P[1], off=P[2], perm=P[3], w=P[4], gu=P[5], dn=P[6], xsh=P[7], xshs=P[8],
             sgu=P[9], sdn=P[10], Y=P[11], Ysh=P[12], ws=P[13],
             nws=fgs.moe_workspace_size(cfg, 4))
    a.update(over)
    return fgs.lib.moe_grouped_swiglu_fp8_rows(
        ctypes.byref(cfg), 4, a["x"], a["xs"], a["off"], a["perm"], a["w"], a["gu"], a["dn"],
        a["xsh"], a["xshs"], a["sgu"], a["sdn"], a["Y"], a["Ysh"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("layout,over,status", [
    (0, {}, 2), (1, {}, 2), (2, {}, 2),          # E4M3 rows need a 4-bit layout
    (3, {"xs": None}, 1), (3, {"xshs": None}, 1), (3, {"Ysh": None}, 1), (3, {"gu": None}, 1),
    (4, {"xs": P[1] + 4}, 3), (4, {"x": P[0] + 1}, 3), (3, {"ws": None}, 4), (3, {"nws": 1024}, 4),
])
def test_fp8_rows_refusals(fgs, layout, over, status):
    assert _swiglu(fgs, layout, **over) == status


@pytest.mark.parametrize("args,status", [
    ((7, 4, 256, P[0], P[1], P[2], 1e-6, P[3], P[4], None, None), 1),     # dtype
    ((1, 0, 256, P[0], P[1], P[2], 1e-6, P[3], P[4], None, None), 1),     # T
    ((1, 4, 0, P[0], P[1], P[2], 1e-6, P[3], P[4], None, None), 1),       # d
    ((1, 4, 256, None, P[1], P[2], 1e-6, P[3], P[4], None, None), 1),
    ((1, 4, 256, P[0], P[1], None, 1e-6, P[3], P[4], None, None), 1),
    ((1, 4, 256, P[0], P[1], P[2], -1.0, P[3], P[4], None, None), 1),     # eps
    ((1, 4, 256, P[0], P[1], P[2], float("nan"), P[3], P[4], None, None), 1),
    ((1, 4, 256, P[0], P[1], P[2], 1e-6, P[3], None, None, None), 1),     # no output
    ((1, 4, 256, P[0], P[1], P[2], 1e-6, P[3], P[4], P[5], None), 1),     # codes without scales
    ((1, 4, 256, P[0], P[1], P[2], 1e-6, P[3], P[4], None, P[6]), 1),
    ((1, 4, 200, P[0], P[1], P[2], 1e-6, P[3], P[4], P[5], P[6]), 2),     # 8 bits: d % 128
    ((1, 4, 256, P[0] + 2, P[1], P[2], 1e-6, P[3], P[4], None, None), 3),
    ((0, 4, 256, P[0], P[1], P[2], 1e-6, P[3], P[4], P[5], P[6] + 4), 3),
])
def test_norm_refusals(fgs, args, status):
    assert fgs.lib.moe_add_rmsnorm(*args, None) == status


def test_binding_raises_with_the_name(fgs):
    with pytest.raises(fgs.MoeError) as e:
        fgs.moe_linear_int4(0, 256, 64, 32, P[0], None, P[1], None, P[2], stream=0)
    assert e.value.status == 1
