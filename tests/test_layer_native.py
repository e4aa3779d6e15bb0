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


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_product_sizes_reach_every_kernel(tmp_path):
    """The sizes that the GPU tests compare with the exact product take, on 256 CUs,
    every kernel of the dispatch: each with K in whole rounds of its buffers and with
    a tail; the few-rows kernels with sums shorter than the pieces under way at a time,
    shorter than twice that, and longer (their main loop); the tiles with last tiles
    shifted in rows and in columns."""
    from tests.test_gpu_layer import MM
    from tests.test_gpu_layer_edges import MM_KERNELS
    repo = os.path.dirname(HERE)
    exe = tmp_path / "kinds"
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{os.path.join(repo, 'mamba_ssd_chunked_amd', 'csrc')}",
                    os.path.join(HERE, "native", "matmul_kinds.cpp"), "-o", str(exe)], check=True, timeout=300)
    sizes = MM + MM_KERNELS
    r = subprocess.run([str(exe)], input="".join(f"{m} {n} {k}\n" for m, n, k in sizes), capture_output=True, text=True,
                       check=True, timeout=60)
    seen = set()
    ahead = {0: 2, 1: 3, 2: 2, 3: 2}  # pieces under way in the few-rows kernels
    for (m, n, k), line in zip(sizes, r.stdout.splitlines()):
        i, rows, cols, rnd = map(int, line.split())
        seen.add((i, "tail" if k % rnd else "whole"))
        if i in ahead:
            pieces = -(-k // rnd)
            seen.add((i, "short" if pieces < ahead[i] else "once" if pieces < 2 * ahead[i] else "loop"))
        else:
            seen |= {(i, "rows")} if m % rows else set()
            seen |= {(i, "columns")} if n % cols else set()
    want = {(i, what) for i in range(7) for what in ("tail", "whole")}
    want |= {(i, what) for i in range(4) for what in ("short", "once", "loop")}
    want |= {(i, what) for i in range(4, 7) for what in ("rows", "columns")}
    want.discard((3, "short"))  # 64 x 64 blocks with K of one piece are never the fastest
    assert want <= seen, sorted(want - seen)
