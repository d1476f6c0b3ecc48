"""Checks of the gfx950 assembly of the gated kernels. Needs hipcc, no GPU."""
import os
import subprocess

import pytest

from tests.test_device_code_cpu import CSRC, _build_module, parse, unordered_exchanges


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{kernel: instructions} of the gated microscaled product, with the library's own flags."""
    mod = _build_module()
    try:
        hipcc = mod._hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    s = str(tmp_path_factory.mktemp("asm") / "mx_gated.s")
    r = subprocess.run([hipcc] + mod._flags() + ["-x", "hip", "-S", "--offload-device-only", os.path.join(CSRC, "mx_gated.hip"), "-o", s],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    return parse(open(s).read())


def test_rows_through_lds_are_ordered(kernels):
    """The tiles bring rows of H together in LDS before they store them: five
    tiles, dense and by expert, and two of them together, two types of X each."""
    names = ("10k_mx_gated", "18k_mx_gated_grouped", "14k_mx_gated_two")
    tiles = {n: k for n, k in kernels.items() if k.code and any(name in n for name in names)}
    assert len(tiles) == 22
    for name, kernel in tiles.items():
        assert any(c.startswith("ds_write") for c in kernel.code), name
        found = unordered_exchanges(kernel)
        assert not found, f"{name}: {len(found)}, first {found[0]}"
