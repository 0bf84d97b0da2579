"""Which matrices overlap, as the entry points' EALIAS has it (host: tests/c/strided.cpp, against the bytes)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_matrices_overlap_where_they_share_a_byte(tmp_path):
    out = str(tmp_path / "strided")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", os.path.join(ROOT, "tests", "c", "strided.cpp"), "-o", out, "-I",
                    os.path.join(ROOT, "fully_sharded_gb300", "csrc"), "-I", os.path.join(ROOT, "include")], check=True)
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
