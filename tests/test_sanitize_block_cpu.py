"""The C ABI layer of qlora_block.h (api_block.cpp, with the checks of api.cpp
and api_mx.cpp that it shares) built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer against host-only stand-ins of the launchers, and
driven through every entry point with invalid and valid arguments. Needs no
GPU."""
import os
import shutil

import pytest

from tests.test_sanitize_cpu import CSRC, FLAGS, HIP, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or shutil.which("gcc") is None, reason="no host compiler")
def test_block_abi_rejections_under_asan_ubsan(tmp_path):
    objs = []
    sources = [os.path.join(CSRC, f"{n}.cpp") for n in ("api", "api_mx", "api_block", "codebook", "profile")]
    sources += [os.path.join(SAN, f"{n}.cpp") for n in ("stubs", "stubs_mx", "stubs_block")]
    for src in sources:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        _run(["g++", "-std=c++17", "-Wall"] + HIP + FLAGS + ["-c", src, "-o", objs[-1]], tmp_path)
    main = str(tmp_path / "reject_block.o")
    _run(["gcc", "-std=c11", "-Wall", "-Werror"] + FLAGS + ["-c", os.path.join(SAN, "reject_block.c"), "-o", main], tmp_path)
    exe = str(tmp_path / "reject_block")
    _run(["g++"] + FLAGS + [main] + objs + ["-o", exe], tmp_path)
    r = _run([exe], tmp_path)
    assert "reject_block: ok" in r.stdout and "runtime error" not in r.stderr, r.stdout + r.stderr
