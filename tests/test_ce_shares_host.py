"""The tile shares of the linear cross entropy's launches, compiled for the host (CPU)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_tile_once_and_level_loads(tmp_path):
    exe = str(tmp_path / "ce_shares_host")
    src = os.path.join(ROOT, "tests", "host", "ce_shares_host.cpp")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fsanitize=undefined,address", "-o", exe, src], check=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout + res.stderr
