"""The walks over a batch that the cache's kernels take, run on the host from the kernels' own headers: every piece of work
of a batch is found once, and cu and seq_lens that hold anything lead to nothing outside it."""
import os
import subprocess

import pytest

from fp8_block_scaled_05_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    exe = str(tmp_path_factory.mktemp("walk") / "kv_walk_check")
    r = subprocess.run([cc, "-x", "hip", "--offload-host-only", "-O2", "-std=c++17", "-fwrapv", "-I", build.INCLUDE, "-I", build.CSRC,
                        os.path.join(HERE, "kv_walk_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


@pytest.mark.parametrize("name", ["tiles", "crooked_tiles", "many_tiles", "slots", "crooked_slots"])
def test_walk(check, name):
    r = subprocess.run([check, name], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout
