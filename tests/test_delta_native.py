"""CPU checks of the gated delta rule's host-readable parts (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mamba_ssd_chunked_amd", "csrc")
FP16_MOST = 65504.0

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


def native(tmp_path, name, stdin=""):
    exe = tmp_path / name
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", os.path.join(HERE, "native", f"{name}.cpp"), "-o", str(exe)],
                   check=True, timeout=300)
    return subprocess.run([str(exe)], input=stdin, capture_output=True, text=True, check=True, timeout=60).stdout


def test_scaled_operands_stay_in_fp16s_range(tmp_path):
    """A scale brings a largest value to [2^8, 2^9), and the largest state that a chunk can leave,
    with keys and changes just below a power of two and of one sign, is a number of fp16."""
    inverse, least, most, scaled, state, bound = map(float, native(tmp_path, "delta_scale").split())
    assert inverse == 1 and least >= 256 and most < scaled == 512
    assert 0.9 * bound < state <= bound < FP16_MOST


def test_steps_fit_a_launch(tmp_path):
    """A launch holds fewer than 2^32 threads, at any number of heads that the calls take."""
    most, whole, *passes = map(int, native(tmp_path, "delta_kind").split())
    assert 2 ** 31 < most < 2 ** 32 and whole
    assert passes == [1, 4, 4, 4, 8]
