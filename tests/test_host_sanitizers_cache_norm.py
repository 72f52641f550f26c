"""The host side of attention over a paged cache, of the calls on a cache in 8 bits and
of the step between two blocks under AddressSanitizer and UndefinedBehaviorSanitizer
(CPU only): which kernel a call takes and how its work is cut, the addresses and strides
it is given, that the workspace holds every plan of its sizes, and the refusals
(tests/host/cache_norm_driver.cpp)."""
import os
import shutil

import pytest

_san = pytest.importorskip("test_host_sanitizers")   # its flags and runner
HOST, ROOT, SAN, _run = _san.HOST, _san.ROOT, _san.SAN, _san._run


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_cache_and_norm_host_code(tmp_path):
    csrc = os.path.join(ROOT, "tensor_linear_amd", "csrc")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", csrc, "-I", "/opt/rocm/include", "-D__HIP_PLATFORM_AMD__"]
    objs = []
    for name in ("tplinear", "tplinear_cache", "tplinear_norm", "attn"):
        objs.append(str(tmp_path / f"{name}.o"))
        _run(["g++", "-std=c++17", "-O1", "-c", os.path.join(csrc, f"{name}.cpp"), "-o", objs[-1]] + SAN + inc, tmp_path)
    exe = str(tmp_path / "driver")
    _run(["g++", "-std=c++17", "-O1", os.path.join(HOST, "cache_norm_driver.cpp"), *objs, "-o", exe] + SAN + inc, tmp_path)
    r = _run([exe], tmp_path)
    assert "cache and norm driver ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
