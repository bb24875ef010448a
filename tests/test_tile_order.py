"""How the tile kernels of the projection and of the log-probabilities deal out their tiles, checked in C++ on the
host (tests/tile_order.cpp)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "prefix_shared_chunkwise_gb300", "csrc")


def test_every_tile_once(tmp_path):
    exe = str(tmp_path / "tile_order")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, os.path.join(ROOT, "tests", "tile_order.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
