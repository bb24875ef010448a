"""The planner's tables of the scan, checked in C++ on the host (tests/scan_tables.cpp)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "prefix_shared_chunkwise_gb300", "csrc")


def test_tables_of_random_forests(tmp_path):
    exe = str(tmp_path / "scan_tables")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "scan_tables.cpp"), os.path.join(CSRC, "plan.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
