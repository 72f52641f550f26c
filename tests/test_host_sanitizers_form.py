"""Which form an attention call takes and how its work is cut (attn.cpp), under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only;
tests/host/attention_form_driver.cpp)."""
import os
import shutil

import pytest

_san = pytest.importorskip("test_host_sanitizers")   # its flags and runner
HOST, ROOT, SAN, _run = _san.HOST, _san.ROOT, _san.SAN, _san._run


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_attention_forms(tmp_path):
    csrc = os.path.join(ROOT, "tensor_linear_amd", "csrc")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", csrc, "-I", "/opt/rocm/include", "-D__HIP_PLATFORM_AMD__"]
    exe = str(tmp_path / "driver")
    _run(["g++", "-std=c++17", "-O1", os.path.join(HOST, "attention_form_driver.cpp"), os.path.join(csrc, "attn.cpp"), "-o", exe] + SAN + inc, tmp_path)
    r = _run([exe], tmp_path)
    assert "attention form driver ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
