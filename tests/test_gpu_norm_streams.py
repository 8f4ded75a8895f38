"""moe_norm_backward of many rows of whole 16-byte chunks, where a block keeps copies of
its next rows under way: every number of blocks an SM has (1 to 16 by the width), with
all threads' chunks in the row and with fewer, in both norms and types, against fp64;
dx in place of each input; some of the outputs."""
import pytest
import torch

from _gpu_common import lib, need_gpu
from test_gpu_layernorm import _backward, _check_backward, _inputs

pytestmark = pytest.mark.gpu

# past the limits up to which rows are read twice: 1536 rows of bf16, 24 MB of rows and
# gradients; 16 blocks an SM from 19456 rows of at most 512 columns on
SHAPES = [(1603, 264), (1700, 512), (2001, 1032), (3100, 1024), (1700, 2056), (3100, 2048), (1601, 4104),
          (1601, 4096), (1543, 8184), (19460, 264), (19460, 512)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_against_fp64(T, d, dtype, kind):
    need_gpu()
    fgs = lib()
    x, r, w, _, dy, g = _inputs(T, d, dtype)
    _check_backward(kind, dtype, x, r, w, dy, g, _backward(fgs, kind, dtype, x, r, w, dy, g))


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1603, 264), (2001, 1032), (3100, 2048), (1601, 4104), (19460, 512)])
def test_in_place(T, d, dtype, kind):
    need_gpu()
    fgs = lib()
    x, r, w, _, dy, dh = (t.cuda() for t in _inputs(T, d, dtype))
    full = _backward(fgs, kind, dtype, x, r, w, dy, dh)
    for at in range(4):
        t = [v.clone() for v in (x, r, dy, dh)]
        got = _backward(fgs, kind, dtype, t[0], t[1], w, t[2], t[3], dx=t[at])
        for name in full:
            assert full[name] is None or torch.equal(got[name], full[name])
        for i, v in enumerate((x, r, dy, dh)):  # and nothing else is written
            assert i == at or torch.equal(t[i], v)
    for want in (("dw",), ("dx", "dw")) + ((("dx", "db"), ("db",)) if kind == "layer" else ()):
        got = _backward(fgs, kind, dtype, x, r, w, dy, dh, want=want)
        for name in want:
            if name == "dx" or "dx" in want:
                assert torch.equal(got[name], full[name])
        if "dx" not in want:  # without dx dh is not read
            other = _backward(fgs, kind, dtype, x, r, w, dy, None, want=want)
            for name in want:
                assert torch.equal(got[name], other[name])
