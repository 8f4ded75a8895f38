"""Refusals of the training operators, which come before any CUDA call."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def fgs():
    import __graft_entry__
    __graft_entry__.build()
    import fine_grained_sparse_gb300 as m
    return m


P = [0x100000 * (i + 1) for i in range(16)]  # aligned addresses, never dereferenced


def _cfg(fgs, **kw):
    base = dict(d_model=256, d_ff=128, E_routed=8, K=2)
    base.update(kw)
    return fgs.config(**base)


@pytest.mark.parametrize("kw,T,args,status", [
    ({}, 0, P[:5], 1),
    ({}, 1 << 31, P[:5], 1),
    ({"K": 9}, 4, P[:5], 1),
    ({"K": 33, "E_routed": 64}, 4, P[:5], 2),
    ({"d_model": 200}, 4, P[:5], 2),
    ({"dtype": 5}, 4, P[:5], 1),
    ({}, 1 << 30, P[:5], 2),                                   # T K
    ({}, 4, [None, P[1], P[2], P[3], P[4]], 1),
    ({}, 4, [P[0], None, P[2], P[3], P[4]], 1),
    ({}, 4, [P[0], P[1], P[2], None, P[4]], 1),
    ({}, 4, [P[0], P[1], P[2], P[3], None], 1),                # weights and no place for them
    ({}, 4, [P[0], P[1], None, P[3], P[4]], 1),
    ({}, 4, [P[0] + 8, P[1], P[2], P[3], P[4]], 3),
    ({}, 4, [P[0], P[1] + 4, P[2], P[3], P[4]], 3),
    ({}, 4, [P[0], P[1], P[2], P[3], P[4] + 4], 3),
])
def test_gather_refusals(fgs, kw, T, args, status):
    assert fgs.lib.moe_gather(ctypes.byref(_cfg(fgs, **kw)), T, *args, None) == status
    assert fgs.lib.moe_gather(None, 4, *P[:5], None) == 1


@pytest.mark.parametrize("kw,T,over,status", [
    ({}, 0, {}, 1),
    ({"d_latent": 100}, 4, {}, 2),
    ({}, 4, {0: None}, 1),                # dy
    ({}, 4, {2: None}, 1),                # inv
    ({}, 4, {4: None, 5: None}, 1),       # no output
    ({}, 4, {1: None}, 1),                # dtopk_w without Y
    ({}, 4, {0: P[0] + 2}, 3),
    ({}, 4, {3: P[3] + 4}, 3),
    ({}, 4, {5: P[5] + 8}, 3),
])
def test_combine_backward_refusals(fgs, kw, T, over, status):
    a = [over.get(i, P[i]) for i in range(6)]
    assert fgs.lib.moe_combine_backward(ctypes.byref(_cfg(fgs, **kw)), T, *a, None) == status


@pytest.mark.parametrize("kw,T,over,status", [
    ({}, 0, {}, 1),
    ({"E_routed": 1025}, 4, {}, 1),
    ({"routed_scaling_factor": math.inf}, 4, {}, 1),
    ({}, 4, {0: None}, 1), ({}, 4, {1: None}, 1), ({}, 4, {2: None}, 1), ({}, 4, {3: None}, 1),
    ({}, 4, {3: P[0]}, 1),                # in place
    ({}, 4, {2: P[2] + 4}, 3), ({}, 4, {3: P[3] + 8}, 3),
])
def test_router_backward_refusals(fgs, kw, T, over, status):
    a = [over.get(i, P[i]) for i in range(4)]
    assert fgs.lib.moe_router_backward(ctypes.byref(_cfg(fgs, **kw)), T, *a, None) == status


@pytest.mark.parametrize("args,status", [
    ((2, 4, 256, P[0], P[1], P[2], P[3], 1e-6, P[4], P[5]), 1),       # dtype
    ((1, 0, 256, P[0], P[1], P[2], P[3], 1e-6, P[4], P[5]), 1),       # T
    ((1, 4, 0, P[0], P[1], P[2], P[3], 1e-6, P[4], P[5]), 1),         # d
    ((1, 4, 256, P[0], P[1], P[2], P[3], math.inf, P[4], P[5]), 1),   # eps
    ((1, 4, 256, None, P[1], P[2], P[3], 1e-6, P[4], P[5]), 1),
    ((1, 4, 256, P[0], P[1], None, P[3], 1e-6, P[4], P[5]), 1),
    ((1, 4, 256, P[0], P[1], P[2], P[3], 1e-6, P[4], None), 1),
    ((1, 4, 256, P[0], P[1], P[2], P[3], 1e-6, P[4], P[4]), 1),       # h and y one buffer
    ((1, 4, 256, P[0], P[1], P[2], P[3] + 2, 1e-6, P[4], P[5]), 3),
    ((0, 4, 256, P[0], P[1], P[2], P[3], 1e-6, P[4] + 4, P[5]), 3),
])
def test_layernorm_refusals(fgs, args, status):
    assert fgs.lib.moe_add_layernorm(*args, None) == status


def _norm_backward(fgs, **over):
    a = dict(kind=1, dtype=1, T=4, d=256, x=P[0], res=None, w=P[1], eps=1e-6, dy=P[2], dh=None,
             dx=P[3], dw=P[4], db=P[5], ws=P[6], nws=fgs.moe_norm_backward_workspace_size(4, 256))
    a.update(over)
    return fgs.lib.moe_norm_backward(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    ({"kind": 2}, 1), ({"dtype": 3}, 1), ({"T": 0}, 1), ({"d": 0}, 1), ({"eps": -1.0}, 1),
    ({"eps": math.nan}, 1), ({"x": None}, 1), ({"w": None}, 1), ({"dy": None}, 1),
    ({"dx": None, "dw": None, "db": None}, 1),
    ({"kind": 0}, 1),                            # an RMS norm has no bias
    ({"x": P[0] + 2}, 3), ({"dh": P[7] + 8}, 3), ({"dw": P[4] + 4}, 3), ({"db": P[5] + 4}, 3),
    ({"ws": None}, 4), ({"nws": 256}, 4), ({"ws": P[6] + 4}, 3),
    ({"T": 5}, 4),                               # a workspace of fewer rows
])
def test_norm_backward_refusals(fgs, over, status):
    assert _norm_backward(fgs, **over) == status


def test_norm_backward_workspace(fgs):
    size = fgs.moe_norm_backward_workspace_size
    assert size(0, 8) == size(4, 0) == size((1 << 30) + 1, 8) == 0
    # a partial row of dweight and one of dbias for every block of rows
    assert size(8192, 7168) >= 2 * 4 * 304 * 7168
    assert size(1, 1) > 0


def _adamw(fgs, tensor=(), n_tensors=1, tensors=True, **over):
    t = dict(param=P[0], grad=P[1], master=P[2], exp_avg=P[3], exp_avg_sq=P[4], exp_avg_scale=P[5],
             exp_avg_sq_scale=P[6], n=1000, weight_decay=0.1)
    t.update(tensor)
    a = dict(pd=1, gd=1, bits=8, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, step=1, gs=None, seed=0)
    a.update(over)
    e = (fgs.AdamwTensor * 1)(fgs.AdamwTensor(**t))
    return fgs.lib.moe_adamw(n_tensors, ctypes.addressof(e) if tensors else None, *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    ({"n_tensors": -1}, 1), ({"tensors": False}, 1), ({"pd": 2}, 1), ({"gd": -1}, 1),
    ({"bits": 16}, 2), ({"lr": -1.0}, 1), ({"lr": math.nan}, 1), ({"b1": 1.0}, 1),
    ({"b2": -0.1}, 1), ({"b2": math.nan}, 1), ({"eps": -1e-8}, 1), ({"eps": math.inf}, 1),
    ({"step": 0}, 1), ({"gs": P[7] + 2}, 3),
    ({"tensor": {"n": -1}}, 1), ({"tensor": {"n": (1 << 40) + 1}}, 1),
    ({"tensor": {"weight_decay": -0.1}}, 1), ({"tensor": {"weight_decay": math.inf}}, 1),
    ({"tensor": {"param": None}}, 1), ({"tensor": {"grad": None}}, 1),
    ({"tensor": {"exp_avg": None}}, 1), ({"tensor": {"exp_avg_sq": None}}, 1),
    ({"tensor": {"exp_avg_scale": None}}, 1), ({"tensor": {"exp_avg_sq_scale": None}}, 1),
    ({"pd": 0}, 1),                              # a master copy of an fp32 param
    ({"bits": 32}, 1),                           # scales of fp32 states
    ({"tensor": {"param": P[0] + 8}}, 3), ({"tensor": {"grad": P[1] + 2}}, 3),
    ({"tensor": {"master": P[2] + 4}}, 3), ({"tensor": {"exp_avg": P[3] + 1}}, 3),
    ({"tensor": {"exp_avg_scale": P[5] + 2}}, 3), ({"tensor": {"exp_avg_sq_scale": P[6] + 1}}, 3),
])
def test_adamw_refusals(fgs, kw, status):
    assert _adamw(fgs, **kw) == status


def test_adamw_of_nothing(fgs):
    """No tensor, or only empty ones, is no work and no error."""
    n = fgs.moe_launch_count()
    assert fgs.lib.moe_adamw(0, None, 1, 1, 8, 1e-3, 0.9, 0.99, 1e-8, 1, None, 0, None) == 0
    assert _adamw(fgs, tensor={"n": 0, "param": None, "grad": None}) == 0
    assert fgs.moe_launch_count() == n


def test_adamw_table_refuses(fgs):
    torch = pytest.importorskip("torch")
    x = torch.zeros(8)
    with pytest.raises(ValueError):  # not on a GPU
        fgs.adamw_table([{"param": x, "grad": x, "exp_avg": x, "exp_avg_sq": x}])
    assert len(fgs.adamw_table([])) == 0


def test_bindings_raise_with_the_name(fgs):
    with pytest.raises(fgs.MoeError, match="moe_norm_backward"):
        fgs.moe_norm_backward(3, 1, 4, 256, P[0], None, P[1], 1e-6, P[2], None, P[3], None, None,
                              stream=0)
    with pytest.raises(fgs.MoeError, match="moe_adamw"):
        fgs.moe_adamw(fgs.adamw_table([]), 1, 1, 8, 1e-3, 2.0, 0.99, 1e-8, 1, stream=0)
