"""Host sanitizer run (AddressSanitizer + UndefinedBehaviorSanitizer) of the norm, INT8 head
and distillation entry points on the CPU.

The C ABI's host code (mosaic_abi_ops.cpp, and mosaic_abi.cpp whose helpers it uses) is built
with hipcc, the sanitizers on its host side only, linked against launcher stand-ins, and driven
through the validation at the edges of int64 and the empty problems
(tests/sanitize/ops_driver.cpp).  Any sanitizer report fails the run.  No GPU is used.
"""
import os

import pytest

from test_sanitize_cpu import ENV, ROOT, SAN, _hipcc, _run


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not found")
def test_ops_abi_host_code_under_asan_ubsan(tmp_path):
    hipcc = _hipcc()
    host_san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                "-Xarch_host", "-fno-sanitize-recover=all"]
    flags = ["-O1", "-g", "-std=c++20", "-I", os.path.join(ROOT, "include"), *host_san]
    csrc = os.path.join(ROOT, "mask_only_logits_amd", "csrc")
    objs = []
    for src, extra in ((os.path.join(csrc, "mosaic_abi.cpp"), ["-x", "hip", "--offload-arch=gfx950"]),
                       (os.path.join(csrc, "mosaic_abi_ops.cpp"), ["-x", "hip", "--offload-arch=gfx950"]),
                       (os.path.join(SAN, "launch_stubs.cpp"), []), (os.path.join(SAN, "ops_stubs.cpp"), []),
                       (os.path.join(SAN, "ops_driver.cpp"), [])):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([hipcc, *extra, *flags, "-c", src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "ops_driver")
    _run([hipcc, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address", "-Xarch_host",
          "-fsanitize=undefined", "-o", exe, *objs])
    assert "ops sanitizer driver ok" in _run([exe], env=ENV)
