"""Checks of the gfx950 assembly that the compiler writes for the library's
own kernels. Needs hipcc, no GPU.

Wait states. The instruction set leaves some distances between instructions to
the program ("manually inserted wait states" of the CDNA ISA documents): one
between a scalar write of M0 and a load into LDS, which takes its address from
it, and five between a vector instruction that writes a scalar register and a
memory instruction that reads it. The compiler inserts them for instructions of
its own but not inside inline assembly, which the copies into LDS are.

Data between lanes. Where lanes of a wave read from LDS what others of the
wave wrote, the hardware keeps the order, but the compiler may only be relied
on to where a barrier, if only the wave's own, stands in between."""
import concurrent.futures
import glob
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_nf4_quantized_03_amd", "csrc")


def _build_module():
    spec = importlib.util.spec_from_file_location("_build_flags", os.path.join(ROOT, "bit_nf4_quantized_03_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    """{source: {kernel: Kernel}} of every .hip source, with the library's own flags."""
    mod = _build_module()
    try:
        hipcc = mod._hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("asm")

    def one(src):
        s = str(out / (os.path.basename(src) + ".s"))
        r = subprocess.run([hipcc] + mod._flags() + ["-x", "hip", "-S", "--offload-device-only", src, "-o", s],
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-4000:]
        return os.path.basename(src), parse(open(s).read())

    with concurrent.futures.ThreadPoolExecutor(4) as ex:
        return dict(ex.map(one, sorted(glob.glob(os.path.join(CSRC, "*.hip")))))


class Kernel:
    def __init__(self):
        self.code, self.labels = [], {}
        self.barriers = []   # the instructions behind the wave's own barriers

    def op(self, k):
        parts = self.code[k].split(None, 1)
        return parts[0], [x.strip() for x in parts[1].split(",")] if len(parts) > 1 else []

    def states(self, k):
        name, args = self.op(k)
        return int(args[0], 0) + 1 if name == "s_nop" else 1

    def before(self):
        """The instructions that may run directly before each one."""
        come = {}
        for k in range(len(self.code)):
            name, args = self.op(k)
            if name.startswith(("s_branch", "s_cbranch")):
                come.setdefault(self.labels[args[0]], []).append(k)
        return [come.get(k, []) + ([k - 1] if k and self.op(k - 1)[0] not in ("s_branch", "s_endpgm") else [])
                for k in range(len(self.code))]

    def closer_than(self, before, k, need, writes):
        """An instruction for which `writes` holds with fewer than `need` wait states between it and number k, or None."""
        todo, seen = [(q, 0) for q in before[k]], set()
        while todo:
            q, between = todo.pop()
            if between >= need or (q, between) in seen:
                continue
            seen.add((q, between))
            if writes(q):
                return q
            todo += [(p, between + self.states(q)) for p in before[q]]
        return None


def parse(text):
    """The functions of an assembly listing, with the places of the barriers."""
    kernels, cur = {}, None
    for line in text.splitlines():
        if cur and line.strip() == "; wave barrier":
            cur.barriers.append(len(cur.code))
        code = line.split(";")[0].rstrip()
        label = re.match(r"([\w.$]+):", code)
        if label and not label[1].startswith(".L"):
            cur = kernels.setdefault(label[1], Kernel())
        elif label and cur:
            cur.labels[label[1]] = len(cur.code)
        elif cur and code.strip() and not code.strip().startswith("."):
            cur.code.append(code.strip())
    return kernels


def scalar_registers(arg):
    m = re.match(r"s(?:\[(\d+):(\d+)\]|(\d+))$", arg)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1)) if m[1] else {int(m[3])}
    return {"vcc"} if arg == "vcc" else set()


def into_lds(code):
    return re.match(r"global_load_lds_", code) or (code.startswith("buffer_load") and code.endswith(" lds"))


def missing_wait_states(kernel):
    found, before = [], kernel.before()
    for k, code in enumerate(kernel.code):
        name, args = kernel.op(k)
        if into_lds(code):
            q = kernel.closer_than(before, k, 1, lambda q: kernel.op(q)[0].startswith("s_") and kernel.op(q)[1][:1] == ["m0"])
            if q is not None:
                found.append((kernel.code[q], code))
        if name.startswith(("global_", "buffer_", "flat_", "scratch_")):
            reads = set().union(*(scalar_registers(a.split()[0]) for a in args if a))

            def writes(q):
                op, dst = kernel.op(q)
                return op.startswith("v_") and any(scalar_registers(d) & reads for d in dst[:2 if "_co_" in op else 1])
            q = kernel.closer_than(before, k, 5, writes) if reads else None
            if q is not None:
                found.append((kernel.code[q], code))
    return found


def unordered_exchanges(kernel):
    """Changes between writing and reading LDS without a barrier in between, from the first write on behind the last
    matrix instruction and the workgroup's last barrier. (What is read in front of it, the sums of other groups of
    waves, lies elsewhere.)"""
    names = [kernel.op(k)[0] for k in range(len(kernel.code))]
    start = max((k for k, n in enumerate(names) if n.startswith("v_mfma") or n == "s_barrier"), default=0)
    found, last, wrote = [], None, False
    for k in range(start, len(names)):
        if k in kernel.barriers:
            last = None
        kind = names[k].startswith(("ds_read", "ds_write")) and names[k][:7]
        if kind:
            if last and last != kind:
                found.append(kernel.code[k])
            last = kind if wrote or kind == "ds_writ" else None
            wrote = wrote or kind == "ds_writ"
    return found


def test_the_check_finds_unordered_exchanges():
    def found(*lines):
        return len(unordered_exchanges(parse("\n".join(("f:", "v_mfma_f32 a0, v0, v1, a0") + lines))["f"]))
    write, read = "ds_write_b64 v0, v[2:3]", "ds_read_b128 v[4:7], v1"
    assert found(write, write, read, read) == 1
    assert found(write, read, write, read) == 3
    assert found(write, "\t; wave barrier", read, "\t; wave barrier", write) == 0
    assert found(read, "s_barrier", read, write, read) == 1
    assert found(write, "s_barrier", read, write, "\t; wave barrier", read) == 0


def test_rows_through_lds_are_ordered(assembly):
    """The large microscaled products bring their rows together in LDS before they store them."""
    kernels = {n: k for n, k in assembly["mx_linear.hip"].items() if "k_mx_gemm" in n and k.code}
    assert len(kernels) == 20
    for name, kernel in kernels.items():
        assert any(c.startswith("ds_write") for c in kernel.code), name
        found = unordered_exchanges(kernel)
        assert not found, f"{name}: {len(found)}, first {found[0]}"


def test_the_check_finds_missing_wait_states():
    load = "global_load_lds_dwordx4 v0, s[4:5]"

    def found(*lines):
        return len(missing_wait_states(parse("\n".join(("f:",) + lines))["f"]))
    assert found("s_mov_b32 m0, s2", load) == 1
    assert found("s_mov_b32 m0, s2", "s_nop 0", load) == 0
    assert found("s_mov_b32 m0, s2", "v_mov_b32 v1, v2", load) == 0
    assert found("s_add_i32 m0, m0, 16", ".LBB0_1:", load, "s_cbranch_scc1 .LBB0_1") == 1
    assert found(".LBB0_1:", load, "s_mov_b32 m0, s2", "s_cbranch_scc1 .LBB0_1") == 0   # the branch lies between
    assert found("v_readfirstlane_b32 s5, v3", "s_nop 3", load) == 1
    assert found("v_readfirstlane_b32 s5, v3", "s_nop 4", load) == 0
    assert found("v_readfirstlane_b32 s6, v3", load) == 0
    assert found("v_cmp_lt_i32_e64 s[4:5], v1, v2", "global_store_dword v0, v1, s[4:5]") == 1


def test_no_missing_wait_states(assembly):
    copies = 0
    for source, kernels in assembly.items():
        for name, kernel in kernels.items():
            copies += sum(bool(into_lds(c)) for c in kernel.code)
            found = missing_wait_states(kernel)
            assert not found, f"{source} {name}: {len(found)}, first {found[0]}"
    assert copies > 0
