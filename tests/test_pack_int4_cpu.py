"""What pack_int4 refuses before it packs: the kernel behind it gets bare
pointers and would read past tensors of other shapes."""
import pytest
import torch


@pytest.fixture(scope="module")
def fgs():
    import __graft_entry__
    __graft_entry__.build()
    import fine_grained_sparse_gb300 as m
    return m


def _codes(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype)


def _scales(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("codes,scales,why", [
    (_codes(1, 16, 2048), _scales(1, 16, 127), "not .1, 16, 2048. and .1, 16, 127."),
    (_codes(1, 16, 2048), _scales(1, 16, 33), "group_size"),
    (_codes(1, 16, 2048), _scales(1, 16, 0), "group_size"),
    (_codes(1, 16, 2048), _scales(1, 15, 128), "group_size"),  # a row short
    (_codes(2, 16, 2048), _scales(1, 16, 128), "group_size"),  # a group short
    (_codes(16, 2048), _scales(16, 128), "group_size"),        # no axis of groups
    (_codes(1, 16, 2048), _scales(16, 128), "group_size"),
    (_codes(1, 16, 2048), _scales(1, 16, 128, dtype=torch.float32), "bfloat16"),
    (_codes(1, 16, 2048), _scales(1, 16, 128, dtype=torch.float16), "bfloat16"),
    (_codes(1, 16, 2048, dtype=torch.int8), _scales(1, 16, 128), "uint8"),
    (_codes(1, 16, 2048, dtype=torch.int32), _scales(1, 16, 128), "uint8"),
    (_codes(1, 16, 2048), _scales(1, 16, 128), "one GPU"),
])
def test_pack_int4_refuses(fgs, codes, scales, why):
    launches = fgs.moe_launch_count()
    with pytest.raises(ValueError, match=why):
        fgs.pack_int4(fgs.MOE_PACK_PLAIN, codes, scales, stream=0)
    assert fgs.moe_launch_count() == launches
