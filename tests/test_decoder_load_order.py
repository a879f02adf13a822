"""Order of the loads in the kernels for few rows by 4-bit and 8-bit weights
that stage whole steps (CPU only, from the built code object).

They have no wait for their copies into LDS: the copies of a step are issued
before its loads into registers, loads arrive in the order of their issue, and
the wait for the weights therefore covers the copies.  So in the prologue and
in each of the loop's two steps every copy has to precede every load.
"""
import re
import subprocess

import pytest

import test_resources as base
from dense_bf16_gemm_amd import build

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def disassemble(d, bundle):
    """{kernel symbol: its instructions as text} of the code object in a bundle."""
    (d / "bundle.bin").write_bytes(bundle)
    subprocess.run([base._tool("clang-offload-bundler"), "--type=o", "--unbundle", f"--input={d / 'bundle.bin'}",
                    f"--output={d / 'co'}", f"--targets=hipv4-amdgcn-amd-amdhsa--{build.ARCH}"],
                   check=True, capture_output=True)
    text = subprocess.run([base._tool("llvm-objdump"), "-d", "--no-show-raw-insn", f"--mcpu={build.ARCH}",
                           str(d / "co")], check=True, capture_output=True, text=True).stdout
    funcs, cur = {}, None
    for line in text.splitlines():
        m = re.match(r"^[0-9a-f]+ <(\S+)>:$", line)
        if m:
            cur = funcs.setdefault(m.group(1), [])
        elif cur is not None and line.startswith("\t"):
            cur.append(line.strip())
    return funcs


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """The kernels of libmm.so's second source (one bundle per source, in order)."""
    d = tmp_path_factory.mktemp("co")
    subprocess.run([base._tool("llvm-objcopy"), "--dump-section", f".hip_fatbin={d / 'fatbin'}", build.LIB],
                   check=True, capture_output=True)
    data = (d / "fatbin").read_bytes()
    starts = [m.start() for m in re.finditer(MAGIC, data)]
    assert len(starts) == len(build.SOURCES)
    return disassemble(d, data[starts[1]:])


def loads_in_order(instructions):
    """One letter per vector memory load: c a copy into LDS, w 16 bytes into
    registers (weights), s fewer (scales and zeros)."""
    out = []
    for text in instructions:
        op = text.split()[0]
        if not op.startswith(("buffer_load", "global_load")):
            continue
        out.append("c" if re.search(r"\blds\b", text) else "w" if op.endswith("dwordx4") else "s")
    return "".join(out)


def in_order(sequence, copies, weights, scales):
    """Prologue and two steps, each all copies and then all loads; what comes
    after the loop copies nothing."""
    step = f"c{{{copies}}}([ws]{{{weights + scales}}})"
    if not re.fullmatch(f"(?:{step}){{3}}[ws]*", sequence):
        return False
    return all(loads.count("w") == weights for loads in re.findall(step, sequence))


def test_in_order_finds_a_late_copy():
    assert in_order("ccwwss" * 3 + "ssw", 2, 2, 2)
    assert in_order("ccswws" * 3, 2, 2, 2)
    assert not in_order("ccwwss" + "cwcwss" + "ccwwss", 2, 2, 2)
    assert not in_order("cwwssc" + "ccwwss" * 2, 2, 2, 2)
    assert not in_order("ccwwss" * 2, 2, 2, 2)


def kernels(code):
    for name, ins in code.items():
        m = re.match(r"_ZN3mmk(?:7gemm_w4|12gemm_q8_rows)ILi(\d+)ELi(\d+)E", name)
        if not m:
            continue
        rows, blocks = int(m.group(1)), int(m.group(2))
        four_bit = "gemm_w4" in name
        if four_bit and rows > 32:  # (half steps, whose waits count loads)
            continue
        copies = rows // 4 if four_bit else max(1, rows // 8)
        yield name, ins, copies, blocks if four_bit else 2 * blocks, 2 if four_bit else 0


def test_copies_of_a_step_precede_its_loads(code):
    checked = 0
    for name, ins, copies, weights, scales in kernels(code):
        sequence = loads_in_order(ins)
        assert in_order(sequence, copies, weights, scales), (name, sequence)
        checked += 1
    assert checked == 27 + 12
