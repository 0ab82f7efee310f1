"""Importing the package, its public names too, loads neither torch nor a library: that is left to the first call."""
import os
import subprocess
import sys

import fp8_block_scaled_05_amd as fb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_star_import_is_light():
    code = ("import sys\nfrom fp8_block_scaled_05_amd import *\nimport fp8_block_scaled_05_amd as fb\n"
            "missing = [n for n in fb.__all__ if n not in globals()]\n"
            "assert not missing, missing\n"
            "assert 'torch' not in sys.modules, 'torch'\n"
            "maps = open('/proc/self/maps').read()\n"
            "assert 'libfp8bs' not in maps and '_marshal' not in maps, 'libraries'\n"
            "try:\n    KVCache(1, 2, 3, 4)\nexcept TypeError as e:\n    assert 'k must be a tensor' in str(e), e\n"
            "else:\n    raise AssertionError('not refused')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_public_names_exist():
    assert all(hasattr(fb, n) for n in fb.__all__) and len(set(fb.__all__)) == len(fb.__all__)
