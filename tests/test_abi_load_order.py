"""Host-only calls before torch is imported leave the process with one HIP runtime: torch's."""
import os
import subprocess
import sys

CODE = """
import bit_weight_only_w4_amd as w4
assert w4.moe_workspace_bytes("nf4_f16", 1, 64, 64, 1, 1) > 0
import os, torch
maps = {l.split()[-1] for l in open("/proc/self/maps") if "libamdhip64" in l}
assert len(maps) == 1, maps
assert os.path.realpath(maps.pop()).startswith(os.path.realpath(os.path.dirname(torch.__file__)))
"""


def test_queries_before_torch():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=100,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]
