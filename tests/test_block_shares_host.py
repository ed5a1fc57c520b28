"""tests/c/share_check.cpp, built with g++ against the training operators'
internal header: two products in one grid share all of its blocks."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_two_products_share_all_blocks(tmp_path):
    exe = str(tmp_path / "share_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "zero_sharded_optimizer_step_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", "share_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[:2000] + r.stderr
    assert "all checks passed" in r.stdout
