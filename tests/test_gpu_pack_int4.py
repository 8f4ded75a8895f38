"""pack_int4 on views and on another stream than the tensors' own."""
import pytest
import torch

from _gpu_common import lib, need_gpu
from _int4_common import bank
from test_gpu_int4 import _gen

pytestmark = pytest.mark.gpu


class _Foreign:
    """A stream of another library: whatever has its handle as cuda_stream."""

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("how", ["stream", "handle", "foreign", "default", "current"])
def test_views_on_another_stream(how):
    """Copies made for the packing and the result belong to the current stream:
    work there before the call is seen, and the copies' memory is not handed out
    again while the other stream reads it."""
    need_gpu()
    fgs = lib()
    q, s = (t.cuda() for t in bank(_gen(9), 24, 2048, 1024, 32))
    want = fgs.pack_int4(fgs.MOE_PACK_GATE_UP, q, s)
    qt, st = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, s))  # same values, a view
    assert not qt.is_contiguous() and not st.is_contiguous()
    late = torch.zeros_like(qt)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # the current stream is behind
    late.copy_(qt)
    stream = {"stream": side, "handle": side.cuda_stream, "foreign": _Foreign(side.cuda_stream),
              "default": 0, "current": None}[how]
    got = fgs.pack_int4(fgs.MOE_PACK_GATE_UP, late, st, stream=stream)
    junk = [torch.full_like(q, 7) for _ in range(4)]  # takes freed memory of that size, if any
    torch.cuda.synchronize()
    assert torch.equal(got, want) and junk[0][0, 0, 0] == 7


@pytest.mark.parametrize("rows,cols,scales,status", [(24, 2048, 64, 2), (16, 96, 3, 1),
                                                     (16, 2048, 32, 2)])
def test_sizes_that_the_library_rejects(rows, cols, scales, status):
    """rows % 16, fewer than 128 columns and 64 columns a scale keep their status."""
    need_gpu()
    fgs = lib()
    q = torch.zeros((1, rows, cols // 2), dtype=torch.uint8, device="cuda")
    s = torch.ones((1, rows, scales), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fgs.MoeError) as e:
        fgs.pack_int4(fgs.MOE_PACK_PLAIN, q, s)
    assert e.value.status == status
