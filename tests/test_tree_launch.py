"""What a tree call asks of the runtime before its launch (no GPU needed: the HIP calls are a recorder's).

The limit of a kernel's dynamic LDS belongs to the kernel, which calls on other threads share: a call that set it to its
own need could lower it between another call's setting and launch.  So every call sets the most that the kernel ever takes."""
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

CALLS = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[2])
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
from rank_state_read_amd import binding as B
at = 1 << 20
for kind in ("gdn", "kda"):
    for qkv in ("bf16", "f32"):
        for V in (64, 80, 96, 112, 128):
            sh = B.make_shape(4, 8, 128, V, 16, 1, 79, 49, kind, qkv, 0)
            for ranks in ([0] * 8, [0, 3, 0, 5, 6, 7, 8, 9]):
                plan = B.Plan(sh, ranks, [0] * 8)
                for nodes in (64, 1, 16, 17, 32, 33, 40, 63, 64):
                    print("call", kind, qkv, V, nodes, flush=True)
                    st = B.lib().sketchssm_tree_read(plan.handle, *[at] * 10, 2, 10, nodes, *[at * (i + 2) for i in range(7)],
                                                     None)
                    assert st == 0, st
"""


@pytest.mark.timeout(120)
def test_the_lds_limit_of_a_kernel_never_falls(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    lib = tmp_path / "recorder.so"
    r = subprocess.run([gcc, "-shared", "-fPIC", "-O1", "-Wall", "-Werror", os.path.join(HERE, "hip_recorder.c"), "-o", str(lib)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([sys.executable, "-c", CALLS, str(lib), os.path.dirname(HERE)], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    limit, call, launches, large = {}, "", 0, 0
    for line in r.stdout.splitlines():
        what, *rest = line.split()
        if what == "call":
            call = line
        elif what == "limit":
            assert limit.setdefault(rest[0], int(rest[2])) == int(rest[2]), call
        else:
            launches += 1
            lds = int(rest[3])
            assert lds <= limit.get(rest[0], 64 * 1024), call
            assert lds <= 160 * 1024, call
            large += lds > 64 * 1024
    assert launches == r.stdout.count("call ") == 2 * 2 * 5 * 2 * 9 and large > 0
