"""CPU check of the layer entry points' host code under sanitizers (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the ROCm headers not available")
def test_layer_host_code_under_address_and_ub_sanitizers(tmp_path):
    """ssd_layer_api.cpp (validation, size arithmetic, weight packing) built for the
    host, every error fatal, linked to launchers that only count."""
    repo = os.path.dirname(HERE)
    csrc = os.path.join(repo, "mamba_ssd_chunked_amd", "csrc")
    exe = tmp_path / "layer_san"
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           f"-I{os.path.join(repo, 'include')}", f"-I{csrc}", os.path.join(csrc, "ssd_layer_api.cpp"),
           os.path.join(HERE, "native", "layer_sanitize.cpp"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert " 0 failures" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
