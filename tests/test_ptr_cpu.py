"""What the binding takes for a pointer, with the library's calls replaced: none of
them runs."""
import pytest


@pytest.fixture
def fgs(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import fine_grained_sparse_gb300 as m

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                raise AssertionError(f"{name} was called with {args}")
            return call
    monkeypatch.setattr(m, "lib", Lib())
    return m


class Buffer:
    def data_ptr(self):
        return 0x7000


def test_pointers(fgs):
    assert fgs._ptr(None) is None
    assert fgs._ptr(0x5000) == 0x5000
    assert fgs._ptr(Buffer()) == 0x7000


@pytest.mark.parametrize("bad", ["x", b"16 bytes or more", True, False, 1.0, [0x5000], bytearray(16),
                                 object()])
def test_refused(fgs, bad):
    """A host object that ctypes would turn into a pointer of its own."""
    with pytest.raises(AttributeError):
        fgs._ptr(bad)
    with pytest.raises(AttributeError):
        fgs.moe_add_layernorm(fgs.MOE_F32, 1, 4, bad, None, 0x1000, None, 1e-6, None, 0x2000, stream=0)
    with pytest.raises(AttributeError):
        fgs.moe_add_rmsnorm(fgs.MOE_F32, 1, 4, 0x1000, None, 0x2000, 1e-6, None, bad, stream=0)
