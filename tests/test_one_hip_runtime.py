"""CPU test: whichever is loaded first, the library and torch share one HIP
runtime.  With two in a process the library's launches fail with 'no
ROCm-capable device'."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import zero_sharded_optimizer_step_amd as Z
%s
import torch
held = {line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}
print(len({p for p in held}), held)
"""


@pytest.mark.parametrize("first", ["Z.lib()", "Z.zero_partition(100, 4, 8)", "Z.zero_xent_workspace_bytes(1, 64, 100)",
                                   "import torch; Z.lib()"])
def test_one_runtime(first):
    r = subprocess.run([sys.executable, "-c", CODE % first], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split()[0] == "1", r.stdout
