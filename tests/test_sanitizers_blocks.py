"""The host-side validation of the block-scaled and grouped calls under
AddressSanitizer and UndefinedBehaviorSanitizer (no GPU): sizes at the ends of
int64, leading dimensions, missing pointers."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "sanitize")
HIPCC = "/opt/rocm/bin/hipcc"
SAN = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all"]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no hipcc")
def test_block_abi_validation_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "abi_blocks_san")
    host_san = []
    for flag in SAN:  # host code only: the device code is not instrumented
        host_san += ["-Xarch_host", flag]
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *host_san,
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "nvfp4_moe_skinny_amd", "csrc"),
                    os.path.join(ROOT, "nvfp4_moe_skinny_amd", "csrc", "api.hip"),
                    os.path.join(HERE, "abi_blocks_main.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)
    # the HIP runtime's own allocations are not the library's: no leak check
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
