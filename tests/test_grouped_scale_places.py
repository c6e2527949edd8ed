"""Where the grouped product finds the MXFP8 scales of a slot in LDS (tests/c/mxfp8_scale_places.cpp), at every depth."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_scale_reads_stay_within_their_row(tmp_path):
    exe = str(tmp_path / "places")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "trellis_quantized_moe_tmoe_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", "mxfp8_scale_places.cpp"), "-o", exe], check=True, capture_output=True, text=True)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and p.stdout.strip() == "PASSED", p.stdout + p.stderr
