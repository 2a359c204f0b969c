"""The library's own machine code: waits that the hardware demands around what
is written in inline assembly, where the compiler does not look (CPU)."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from nvfp4_block_scaled_03_amd import _lib

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{kernel: its instructions and labels ("L3:")} of the library's code objects."""
    if not os.path.exists(_lib.LIB_PATH) or not os.path.exists(OBJDUMP):
        pytest.skip("library not built, or no llvm-objdump")
    d = tmp_path_factory.mktemp("code")
    lib = shutil.copy(_lib.LIB_PATH, d / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", str(lib)], check=True, capture_output=True, cwd=d)
    files = sorted(glob.glob(str(d / "*gfx950")))
    assert files
    out = {}
    for f in files:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--symbolize-operands", f], check=True,
                              capture_output=True, text=True).stdout
        code = None
        for line in text.splitlines():
            line = line.split("//")[0].strip()
            m = re.match(r"(?:[0-9a-f]+ )?<(\w+)>:$", line)
            if m and re.match(r"L\d+$", m[1]):
                code.append(m[1] + ":")
            elif m:
                code = out[os.path.basename(f) + " " + m[1]] = []
            elif line and code is not None:
                code.append(line)
    return out


def _registers(operand):
    """Scalar registers that an operand names."""
    operand = operand.strip()
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    return {operand} if re.match(r"(s\d+|m0|vcc)$", operand) else set()


def _written(instruction):
    """The first operand of an instruction that writes one."""
    parts = instruction.split(None, 1)
    return _registers(parts[1].split(",")[0]) if len(parts) == 2 else set()


def _is_direct_load(instruction):
    return instruction.startswith("global_load_lds") or (
        instruction.startswith(("buffer_load", "global_load")) and instruction.split()[-1] == "lds")


def test_direct_loads_wait_for_the_lds_address(kernels):
    """M0 is read by a direct load into LDS one wait state after a scalar write at
    the earliest, scalar operands five after a vector instruction's write."""
    loads, early = 0, []
    for code in kernels.values():
        code = [line for line in code if not line.endswith(":")]
        for i, line in enumerate(code):
            if not _is_direct_load(line):
                continue
            loads += 1
            if code[i - 1].startswith("s_") and "m0" in _written(code[i - 1]):
                early.append(code[i - 1:i + 1])
            reads = set().union(*(_registers(o.split()[0]) for o in line.split(None, 1)[1].split(","))) | {"m0"}
            waited, j = 0, i - 1
            while waited < 5 and j >= 0:
                if code[j].startswith("v_") and _written(code[j]) & reads:
                    early.append(code[j:i + 1])
                m = re.match(r"s_nop (\w+)", code[j])
                waited += int(m[1], 0) + 1 if m else 1
                j -= 1
    assert loads > 0
    assert not early, f"{len(early)} of {loads} loads, e.g. {early[:3]}"


def _blocks(code):
    """(label or None, instructions) runs; a branch ends its run."""
    out = [[None, []]]
    for line in code:
        if line.endswith(":"):
            out.append([line[:-1], []])
            continue
        out[-1][1].append(line)
        if line.startswith(("s_branch", "s_cbranch", "s_endpgm")):
            out.append([None, []])
    return out


def _outstanding_at_barriers(code):
    """Most LDS accesses that a wavefront may have outstanding at each barrier:
    data flow over its branches, where a wait for n leaves n at most."""
    blocks = _blocks(code)
    at = {label: i for i, (label, _) in enumerate(blocks) if label}
    entry = [-1] * len(blocks)
    entry[0] = 0
    work, found = [0], {}
    while work:
        i = work.pop()
        n, following = entry[i], [i + 1] if i + 1 < len(blocks) else []
        for k, line in enumerate(blocks[i][1]):
            name = line.split()[0]
            if name.startswith("ds_"):
                n = min(n + 1, 16)
            elif name == "s_waitcnt":
                m = re.search(r"lgkmcnt\((\d+)\)", line)
                n = min(n, int(m[1])) if m else n
            elif name == "s_barrier":
                found[(i, k)] = max(n, found.get((i, k), 0))
            elif name == "s_branch":
                following = [at[line.split()[1]]]
            elif name.startswith("s_cbranch"):
                following = following + [at[line.split()[1]]]
            elif name == "s_endpgm":
                following = []
        for j in following:
            if n > entry[j]:
                entry[j] = n
                work.append(j)
    return found


def test_no_lds_access_is_outstanding_at_a_barrier(kernels):
    """What stands behind a barrier may write what was read in front of it."""
    barriers, open_ = 0, {}
    for name, code in kernels.items():
        found = _outstanding_at_barriers(code)
        barriers += len(found)
        if any(found.values()):
            open_[name] = max(found.values())
    assert barriers > 0
    assert not open_, open_


def test_the_reading_of_barriers():
    """A loop whose last read is awaited only behind the barrier of the next trip."""
    trip = ["L0:", "s_waitcnt vmcnt(6)", "s_barrier", "s_waitcnt lgkmcnt(0)", "ds_read_b128 v[0:3], v4", "s_cbranch_scc1 L0",
            "s_endpgm"]
    assert list(_outstanding_at_barriers(trip).values()) == [1]
    trip[1] = "s_waitcnt vmcnt(6) lgkmcnt(0)"
    assert list(_outstanding_at_barriers(trip).values()) == [0]
