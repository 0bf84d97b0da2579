"""The norm's vector loads stay inside the rows (host: the kernel's own index arithmetic, tests/c/row_loads.cpp)."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fully_sharded_gb300", "csrc")


def test_every_load_holds_an_element_of_its_row(tmp_path):
    out = str(tmp_path / "row_loads")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", os.path.join(ROOT, "tests", "c", "row_loads.cpp"), "-o", out, "-I", CSRC],
                   check=True)
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_the_kernels_ask_by_it():
    """Both kernels give a row past the last one cols = 0, and the loads go by holds_some alone."""
    source = open(os.path.join(CSRC, "rmsnorm.cu")).read()
    assert len(re.findall(r"const int cols = row < p\.a\.rows \? all : 0;", source)) == 2
    body = source[source.index("struct RowLoad"):]
    body = body[:body.index("void take(")]
    assert body.count("holds_some<kMap>(") == 2 and "raw[k].load(p + j, first," in body
