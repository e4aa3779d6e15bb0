"""CPU check of the operators' host code under sanitizers (no GPU needed), and of which
kernels the tests' products reach."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
REPO = os.path.dirname(HERE)
CSRC = os.path.join(REPO, "mamba_ssd_chunked_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the ROCm headers not available")
def test_operators_host_code_under_address_and_ub_sanitizers(tmp_path):
    """ssd_operators_api.cpp (validation, size arithmetic) built for the host, every
    error fatal, linked to launchers that only count."""
    exe = tmp_path / "operators_san"
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           f"-I{os.path.join(REPO, 'include')}", f"-I{CSRC}", os.path.join(CSRC, "ssd_operators_api.cpp"),
           os.path.join(HERE, "native", "operators_sanitize.cpp"), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert " 0 failures" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_product_sizes_reach_every_kernel(tmp_path):
    """The aligned products of the GPU tests take, on 256 CUs, every kernel of the 16-bit
    dispatch: each with rows in whole rounds of its buffers and with a tail; the tiles with
    last tiles shifted in rows and in columns, in place among them."""
    from tests.test_gpu_matmul import CASES, KERNELS
    exe = tmp_path / "kinds"
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", os.path.join(HERE, "native", "matmul_kinds.cpp"), "-o", str(exe)],
                   check=True, timeout=300)
    cases = [c for c in CASES + KERNELS if c[3] != "fp32" and c[2] % 8 == 0 and c[8] % 8 == 0]
    r = subprocess.run([str(exe)], input="".join(f"{m} {n} {2 * k}\n" for m, n, k, *_ in cases), capture_output=True,
                       text=True, check=True, timeout=60)
    seen = set()
    for (m, n, k, _, _, _, _, res, _), line in zip(cases, r.stdout.splitlines()):
        i, rows, cols, rnd = map(int, line.split())
        seen.add((i, "tail" if 2 * k % rnd else "whole"))
        if i > 3 and res:
            seen |= {(i, "rows")} if m % rows else set()
            seen |= {(i, "columns")} if n % cols else set()
    want = {(i, what) for i in range(7) for what in ("tail", "whole")}
    want |= {(i, what) for i in range(4, 7) for what in ("rows", "columns")}
    assert want <= seen, sorted(want - seen)
