"""Code-generation checks of the decoder-layer operators' kernels, the second
source of libmm.so (CPU only): LDS and registers within the GPU's, spills
within a recorded budget, no scratch access in any loop of MFMAs, the loads
that the 4-bit kernel's counted waits rely on, and no packed fp32 instruction.
"""
import re
import subprocess

import pytest

import test_resources as base
from dense_bf16_gemm_amd import build

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"

# Kernels with values in scratch, at most this many dwords per lane: the 256 x
# 256 tile's epilogue beside its 256 sums, and the norm gradient that holds a
# row of up to 32768 fp32 values and the sums of its columns at once.
SPILL_BUDGET = {r"gemm_q8_tileILi4ELi4ELi3ELi2ELb0E": 8, r"rms_norm_gradILb1ELi4ELb0E": 56}


@pytest.fixture(scope="module")
def remarks():
    r = build.resource_usage(build.REMARKS_DECODER)
    assert r, "no kernels in the resource remarks"
    return r


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """{kernel symbol: [(address, mnemonic, branch target or None)]} of the
    second code object of libmm.so (one bundle per source, in order)."""
    d = tmp_path_factory.mktemp("co")
    fatbin = d / "fatbin.bin"
    subprocess.run([base._tool("llvm-objcopy"), "--dump-section", f".hip_fatbin={fatbin}", build.LIB],
                   check=True, capture_output=True)
    data = fatbin.read_bytes()
    starts = [m.start() for m in re.finditer(MAGIC, data)]
    assert len(starts) == len(build.SOURCES)
    bundle, co = d / "bundle.bin", d / "gfx950.co"
    bundle.write_bytes(data[starts[1]:])
    subprocess.run([base._tool("clang-offload-bundler"), "--type=o", "--unbundle", f"--input={bundle}",
                    f"--output={co}", f"--targets=hipv4-amdgcn-amd-amdhsa--{build.ARCH}"],
                   check=True, capture_output=True)
    text = subprocess.run([base._tool("llvm-objdump"), "-d", f"--mcpu={build.ARCH}", str(co)],
                          check=True, capture_output=True, text=True).stdout
    head = re.compile(r"^([0-9a-f]+) <(\S+)>:$")
    insn = re.compile(r"^\s+(\S+).*//\s*([0-9A-Fa-f]+):[0-9A-Fa-f ]*(?:<(\S+?)(?:\+0x([0-9a-f]+))?>)?\s*$")
    funcs, entry, cur = {}, {}, None
    for line in text.splitlines():
        m = head.match(line)
        if m:
            cur = m.group(2)
            entry[cur] = int(m.group(1), 16)
            funcs[cur] = []
            continue
        m = insn.match(line)
        if cur is None or not m:
            continue
        target = None
        if m.group(1).startswith(("s_branch", "s_cbranch")) and m.group(3) in entry:
            target = entry[m.group(3)] + int(m.group(4) or "0", 16)
        funcs[cur].append((int(m.group(2), 16), m.group(1), target))
    return funcs


def test_remarks_match_the_built_code_object(remarks, code):
    assert set(remarks) == {k for k in code if k.startswith("_ZN3mmk")}


def test_lds_registers_and_stack(remarks):
    for name, r in remarks.items():
        assert r["LDS Size [bytes/block]"] <= base.LDS_MAX, name
        assert r.get("Dynamic Stack", 0) == 0, name
        assert r["VGPRs"] + r["AGPRs"] <= base.REG_FILE, name


def test_spills_within_budget(remarks):
    for name, r in remarks.items():
        budget = next((v for k, v in SPILL_BUDGET.items() if re.search(k, name)), 0)
        assert r["VGPRs Spill"] <= budget and r["ScratchSize [bytes/lane]"] <= 4 * budget, (name, r)


def test_no_scratch_in_mfma_loops(code):
    checked = 0
    for name, ins in code.items():
        if not any(base._is_mfma(m) for (_, m, _) in ins):
            continue
        loops = base._k_loops(ins)
        assert loops, f"{name}: no K loop found"
        for body in loops:
            assert not any(m.startswith("scratch_") for m in body), name
        checked += 1
    assert checked >= 20


def test_no_packed_fp32(code):
    for name, ins in code.items():
        assert not any(re.match(r"v_pk_(add|mul|fma)_f32", m) for (_, m, _) in ins), name


def test_w4_half_steps_issue_the_loads_their_waits_count(code):
    """48 and 64 rows: a wave's waits leave in flight the loads issued after
    the half they wait for, NB blocks of weights, the scales and the zeros, and
    XR / 8 copies per half; the loop (two steps) has to issue exactly those."""
    checked = 0
    for name, ins in code.items():
        m = re.match(r"_ZN3mmk7gemm_w4ILi(48|64)ELi(\d)E", name)
        if not m:
            continue
        xr, nb = int(m.group(1)), int(m.group(2))
        for body in base._k_loops(ins):
            loads = sum(i.startswith(("global_load", "buffer_load")) for i in body)
            mfma = sum(base._is_mfma(i) for i in body)
            per_step = 4 * (xr // 16) * (nb + 1)
            assert mfma % per_step == 0 and mfma, name
            assert loads == mfma // per_step * (nb + 2 + 2 * (xr // 8)), (name, loads, mfma)
            checked += 1
    assert checked >= 18
