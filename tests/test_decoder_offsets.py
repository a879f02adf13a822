"""Addresses of the 4-bit product's copies, walked on the host (CPU only)."""
import os
import subprocess

from dense_bf16_gemm_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_w4_copies_stay_within_the_activations(tmp_path):
    exe = str(tmp_path / "w4_offsets")
    subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "-I", build.CSRC, "-o", exe,
                    os.path.join(HERE, "c", "w4_offsets.hip")], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
