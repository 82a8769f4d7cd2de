"""Host code of the operators on microscaled 4-bit numbers
(csrc/layer/kda_mx4_api.hip) under AddressSanitizer and UndefinedBehaviorSanitizer
(CPU only; see test_sanitizers.py)."""
from __future__ import annotations

import glob
import os

import pytest

from test_sanitizers import BUILD, CSRC, ENV, ROOT, SAN, _run


def test_mx4_host_code_under_sanitizers(tmp_path):
    from gated_delta_rule_tok_amd import build as B
    hipcc = B.hipcc()
    clang = os.path.join(os.path.dirname(os.path.realpath(hipcc)), "..", "llvm", "bin", "clang")
    if not os.path.exists(clang):
        clang = "/opt/rocm/llvm/bin/clang"
    others = [o for o in sorted(glob.glob(os.path.join(BUILD, "*.hip.o"))) if not o.endswith("kda_mx4_api.hip.o")]
    if not os.path.exists(clang) or len(others) < 5:
        pytest.skip("the library's objects are not built (python -m gated_delta_rule_tok_amd.build)")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    api = str(tmp_path / "mx4_api_san.o")
    _run([hipcc, f"--offload-arch={B.ARCH}", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
          *san, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c",
          os.path.join(CSRC, "layer", "kda_mx4_api.hip"), "-o", api])
    drv = str(tmp_path / "mx4_checks.o")
    _run([clang, "-std=c11", "-O1", "-g", "-fsanitize=address,undefined",
          "-I", os.path.join(ROOT, "include"), "-c", os.path.join(SAN, "mx4_checks.c"), "-o", drv])
    exe = str(tmp_path / "mx4_checks")
    _run([hipcc, f"--offload-arch={B.ARCH}", *san, api, drv, *others, "-o", exe])
    r = _run([exe], env=ENV)
    assert "0 failures" in r.stdout
