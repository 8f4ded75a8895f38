"""The status word of calls without a workspace (moe_linear_int4)."""
import torch

import pytest

from _gpu_common import lib, need_gpu
from test_gpu_int4 import _gen, _rows
from _int4_common import bank


def test_status_word_refuses_null():
    import __graft_entry__
    __graft_entry__.build()
    assert lib().lib.moe_status_word(None) == 1  # MOE_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("rows8", [False, True])
def test_linear_has_a_status(rows8):
    """A call whose waits end leaves the word alone, whatever it holds; one that
    expires is read from it like a workspace's."""
    need_gpu()
    fgs = lib()
    gen = _gen(1)
    q, s = bank(gen, 1, 272, 256, 32)
    x, xs, _ = _rows(gen, 50, 256, rows8)
    W = fgs.pack_int4(fgs.MOE_PACK_PLAIN, q.cuda(), s.cuda())
    y = torch.empty((50, 272), dtype=torch.bfloat16, device="cuda")
    word = fgs.moe_status_word()
    assert word == fgs.moe_status_word()
    assert fgs.moe_get_device_status(word) == 0
    fgs.moe_linear_int4(50, 256, 272, 32, x, xs, W, None, y)
    assert fgs.moe_get_device_status(word) == 0
    first = y.clone()
    fgs.moe_selftest_bounded_wait(word)
    fgs.moe_linear_int4(50, 256, 272, 32, x, xs, W, None, y)
    assert fgs.moe_get_device_status(word) == 6  # MOE_ERR_TIMEOUT, until it is read
    assert fgs.moe_get_device_status(word) == 0
    assert torch.equal(y, first)
