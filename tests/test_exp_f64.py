"""The routing scores' fp64 exponential against the C library's long double one,
on the host."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mxfp4_weight_streaming_amd", "csrc")


def test_exponential_is_an_fp64_evaluation(tmp_path):
    exe = tmp_path / "exp_f64_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-fno-fast-math", "-I", CSRC, "-o", str(exe),
                    os.path.join(HERE, "exp_f64_check.cpp"), "-lm"], check=True)
    r = subprocess.run([str(exe), "4000000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert "points 4000000" in r.stdout
