"""The int8 codes' fast quotient against the correctly rounded division, on the
host: every bf16 value up to the row's amax, for a stride of bf16 amax values
(INT8_QUOTIENT_STRIDE, default 9; 1 checks every amax, about 30 s)."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_int8_quotient_matches_division(tmp_path):
    exe = tmp_path / "int8_quotient_check"
    subprocess.run(["gcc", "-O2", "-std=c11", "-ffp-contract=off", "-fno-fast-math", "-o", str(exe),
                    os.path.join(HERE, "int8_quotient_check.c"), "-lm"], check=True)
    stride = os.environ.get("INT8_QUOTIENT_STRIDE", "9")
    r = subprocess.run([str(exe), stride], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert "mismatches 0" in r.stdout and int(r.stdout.split()[1]) > 10_000_000, r.stdout
