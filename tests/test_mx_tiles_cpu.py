"""The tile rule of the microscaled products (mx_tiles.h), built with g++ and
asked for every power of two and its neighbours that the entry points take:
the launch has to stay below 2^32 threads. Needs no GPU."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_every_launch_fits(tmp_path):
    exe = str(tmp_path / "mx_tiles")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", os.path.join(HERE, "cdiv", "mx_tiles.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and " 0 over" in r.stdout, r.stdout
