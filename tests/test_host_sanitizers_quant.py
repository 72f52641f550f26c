"""The host side of the 8-bit layers and the head steps under AddressSanitizer
and UndefinedBehaviorSanitizer (CPU only): which kernel a call takes for a GPU of
256 CUs, the addresses and strides it is given, and every refusal
(tests/host/quant_heads_driver.cpp)."""
import os
import shutil

import pytest

_san = pytest.importorskip("test_host_sanitizers")   # its flags and runner
HOST, ROOT, SAN, _run = _san.HOST, _san.ROOT, _san.SAN, _san._run


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_quant_and_heads_host_code(tmp_path):
    csrc = os.path.join(ROOT, "tensor_linear_amd", "csrc")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", csrc, "-I", "/opt/rocm/include", "-D__HIP_PLATFORM_AMD__"]
    objs = []
    for name in ("tplinear", "tplinear_quant", "tplinear_heads"):
        objs.append(str(tmp_path / f"{name}.o"))
        _run(["g++", "-std=c++17", "-O1", "-c", os.path.join(csrc, f"{name}.cpp"), "-o", objs[-1]] + SAN + inc, tmp_path)
    exe = str(tmp_path / "driver")
    _run(["g++", "-std=c++17", "-O1", os.path.join(HOST, "quant_heads_driver.cpp"), *objs, "-o", exe] + SAN + inc, tmp_path)
    r = _run([exe], tmp_path)
    assert "quant and heads driver ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
