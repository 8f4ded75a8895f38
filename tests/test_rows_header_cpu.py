"""rows.cuh's load and store take one value or 16 bytes: another number, which would
read or write past the values, does not compile."""
import os
import subprocess

import pytest

CALL = {"load": "auto v = fgs::load<{n}>(p); q[0] = v.v[0];",
        "store": "const float v[{n}] = {{}}; fgs::store<{n}>(p, v); q[0] = v[0];"}


@pytest.mark.parametrize("type_,n,fits", [("__nv_bfloat16", 2, False), ("__nv_bfloat16", 4, False),
                                          ("float", 2, False), ("float", 8, False),
                                          ("__nv_bfloat16", 8, True), ("float", 4, True)])
@pytest.mark.parametrize("call", ["load", "store"])
def test_sizes(call, type_, n, fits, tmp_path):
    import __graft_entry__
    b = __graft_entry__._build_module()
    src = tmp_path / "t.cu"
    src.write_text('#include "rows.cuh"\n__global__ void k(' + type_ + "* p, float* q) { "
                   + CALL[call].format(n=n) + " }\n")
    r = subprocess.run([b.nvcc(), *b.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", b.INCLUDE,
                        "-I", b.CSRC, "-c", str(src), "-o", os.devnull], capture_output=True, text=True)
    assert (r.returncode == 0) == fits, r.stdout + r.stderr
    assert fits or "one value or 16 bytes" in r.stdout + r.stderr
