"""What adamw_table and moe_adamw refuse, on stand-ins for tensors on a GPU: nothing
is read, written or launched."""
import pytest


@pytest.fixture
def fgs():
    import __graft_entry__
    __graft_entry__.build()
    import fine_grained_sparse_gb300 as m
    return m


class Fake:
    """A tensor on a GPU as far as a table looks at it."""
    is_cuda = True
    device = "cuda:0"
    SIZE = {"float32": 4, "bfloat16": 2, "uint8": 1, "float8_e4m3fn": 1, "float16": 2, "float64": 8,
            "int32": 4}
    where = 0x10000

    def __init__(self, n, dtype="float32", at=None):
        self.n, self.dtype = n, "torch." + dtype
        self.at = Fake.where if at is None else at
        Fake.where = max(Fake.where, self.at + n * self.SIZE[dtype] + 255 & ~255)

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def element_size(self):
        return self.SIZE[self.dtype[6:]]

    def data_ptr(self):
        return self.at


def _entry(size=1000, p="float32", g="float32", bits=32, copy=False, **over):
    state = "uint8" if bits == 8 else "float32"
    e = {"param": Fake(size, p), "grad": Fake(size, g), "exp_avg": Fake(size, state),
         "exp_avg_sq": Fake(size, state)}
    if copy:
        e["master"] = Fake(size)
    if bits == 8:
        e["exp_avg_scale"], e["exp_avg_sq_scale"] = Fake(-(-size // 128)), Fake(-(-size // 128))
    e.update(over)
    return e


def test_types_of_a_table(fgs):
    assert fgs.adamw_table([]).types == (None, None, None)
    assert fgs.adamw_table([_entry(), _entry(5)]).types == (fgs.MOE_F32, fgs.MOE_F32, 32)
    t = fgs.adamw_table([_entry(p="bfloat16", bits=8, copy=True)])
    assert t.types == (fgs.MOE_BF16, fgs.MOE_F32, 8)
    t = fgs.adamw_table([_entry(bits=8, exp_avg=Fake(1000, "float8_e4m3fn"))])
    assert t.types[2] == 8
    # nothing is done for an empty tensor, whatever it is
    assert fgs.adamw_table([_entry(0, p="float16"), _entry()]).types[0] == fgs.MOE_F32


@pytest.mark.parametrize("over", [{"param": "float16"}, {"param": "float64"}, {"grad": "float16"},
                                  {"exp_avg": "bfloat16"}, {"exp_avg_sq": "int32"},
                                  {"exp_avg": "uint8"}, {"exp_avg_sq": "uint8"},
                                  {"master": "bfloat16"}, {"exp_avg_scale": "bfloat16"}])
def test_table_refuses_types(fgs, over):
    (name, dtype), = over.items()
    with pytest.raises(ValueError, match=name):
        fgs.adamw_table([_entry(**{name: Fake(1000, dtype)})])


@pytest.mark.parametrize("two", [dict(p="bfloat16"), dict(g="bfloat16"), dict(bits=8)])
def test_table_refuses_mixed_types(fgs, two):
    with pytest.raises(ValueError, match="beside others"):
        fgs.adamw_table([_entry(), _entry(**two)])


@pytest.mark.parametrize("entry,args", [
    (dict(p="bfloat16"), ("MOE_F32", "MOE_F32", 32)),   # written past its end
    (dict(), ("MOE_BF16", "MOE_F32", 32)),
    (dict(g="bfloat16"), ("MOE_F32", "MOE_F32", 32)),    # read past its end
    (dict(bits=8), ("MOE_F32", "MOE_F32", 32)),
    (dict(bits=32), ("MOE_F32", "MOE_F32", 8)),
])
def test_call_refuses_other_types(fgs, monkeypatch, entry, args):
    class Lib:
        def __getattr__(self, name):
            raise AssertionError(name + " was called")
    table = fgs.adamw_table([_entry(**entry)])
    monkeypatch.setattr(fgs, "lib", Lib())
    p, g, bits = getattr(fgs, args[0]), getattr(fgs, args[1]), args[2]
    with pytest.raises(ValueError, match="types"):
        fgs.moe_adamw(table, p, g, bits, 1e-3, 0.9, 0.95, 1e-8, 1, stream=0)


def test_table_refuses_overlaps(fgs):
    """A buffer that reaches into one that is written, at any of its elements."""
    base = 0x4000000
    one = _entry(param=Fake(1000, at=base))
    for off in (0, 4, 16, 3996, -4, -3996):
        for name in ("param", "exp_avg", "exp_avg_sq", "grad"):
            with pytest.raises(ValueError, match="already"):
                fgs.adamw_table([one, _entry(**{name: Fake(1000, at=base + off)})])
            with pytest.raises(ValueError, match="already"):
                fgs.adamw_table([_entry(**{name: Fake(1000, at=base + off)}), one])
    for off in (4000, -4000):  # beside it
        fgs.adamw_table([one, _entry(param=Fake(1000, at=base + off))])
    # a large buffer over small ones, and one that only n keeps apart
    with pytest.raises(ValueError, match="already"):
        fgs.adamw_table([one, _entry(100_000, exp_avg=Fake(100_000, at=base - 40_000))])
    fgs.adamw_table([_entry(param=Fake(9000, at=base), n=1000), _entry(8000, param=Fake(8000, at=base + 4000))])
    # gradients are only read: two tensors may have one
    g = Fake(1000)
    fgs.adamw_table([_entry(grad=g), _entry(grad=g)])
    with pytest.raises(ValueError, match="already"):
        fgs.adamw_table([_entry(bits=8, exp_avg_scale=Fake(8, at=base + 64)), _entry(
            bits=8, exp_avg_sq_scale=Fake(8, at=base + 80))])


def test_set_grads(fgs):
    a, b = _entry(), _entry(300)
    t = fgs.adamw_table([a, b, _entry(0)])
    assert [e.grad for e in t.entries][:2] == [a["grad"].at, b["grad"].at]
    g = [Fake(1000), Fake(301), None]
    t.set_grads(g)
    assert [e.grad for e in t.entries] == [g[0].at, g[1].at, None]
    assert t.grads == g and a["grad"] not in t.tensors  # the old ones are let go
    assert [e.param for e in t.entries][:2] == [a["param"].at, b["param"].at]
    beside = Fake(300, at=b["param"].at + 1200)
    t.set_grads((Fake(1000), beside, None))
    t.set_grads([beside_both := Fake(1000), beside_both, None])  # read twice
    fgs.adamw_table([]).set_grads([])


@pytest.mark.parametrize("bad", ["few", "many", "none", "small", "type", "cpu", "device", "strided",
                                 "written"])
def test_set_grads_refuses(fgs, bad):
    a, b = _entry(), _entry(300)
    t = fgs.adamw_table([a, b])
    g = [Fake(1000), Fake(300)]
    if bad == "few":
        g.pop()
    elif bad == "many":
        g.append(Fake(1))
    elif bad == "none":
        g[1] = None
    elif bad == "small":
        g[1] = Fake(299)
    elif bad == "type":
        g[1] = Fake(600, "bfloat16")
    elif bad == "cpu":
        g[1].is_cuda = False
    elif bad == "device":
        g[1].device = "cuda:1"
    elif bad == "strided":
        g[1].is_contiguous = lambda: False
    else:
        for name in ("param", "exp_avg", "exp_avg_sq"):
            for off in (0, 1196, -1196):
                with pytest.raises(ValueError, match="set_grads"):
                    t.set_grads([g[0], Fake(300, at=b[name].at + off)])
        g[1] = Fake(300, at=a["exp_avg"].at + 2000)
    with pytest.raises(ValueError, match="set_grads"):
        t.set_grads(g)
    assert [e.grad for e in t.entries] == [a["grad"].at, b["grad"].at]
    assert t.grads == [a["grad"], b["grad"]]


def test_seed_of_a_step(fgs, monkeypatch):
    """Without one the step's number: random roundings differ from step to step."""
    seen = []

    class Lib:
        def moe_adamw(self, *args):
            seen.append(args)
            return 0
    monkeypatch.setattr(fgs, "lib", Lib())
    for step in (1, 2, 1000):
        fgs.moe_adamw(fgs.adamw_table([]), 1, 1, 8, 1e-3, 0.9, 0.95, 1e-8, step, stream=0)
    fgs.moe_adamw(fgs.adamw_table([]), 1, 1, 8, 1e-3, 0.9, 0.95, 1e-8, 7, None, 0, 0)
    fgs.moe_adamw(fgs.adamw_table([]), 1, 1, 8, 1e-3, 0.9, 0.95, 1e-8, 7, seed=55, stream=0)
    assert [a[11] for a in seen] == [1, 2, 1000, 0, 55]
