"""Loads to LDS that are written in asm, in the assembly of the kernels that have them (hipcc on the host, no GPU). The compiler does
not see what such a load reads: a scalar register that a vector instruction wrote (v_readlane, v_readfirstlane) needs five wait states
before a load may take its address from it, and m0, the LDS address, must stay as the asm set it. Without the wait states a
load once went to another address."""
import importlib.util
import os
import re
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "bit_plane_weight_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def scalar_registers(text):
    out = set()
    for m in re.finditer(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        out |= {int(m.group(3))} if m.group(3) else set(range(int(m.group(1)), int(m.group(2)) + 1))
    return out


def hazards(asm):
    """Loads to LDS, those of them whose scalar operands a vector instruction wrote fewer than five wait states before, and
    instructions outside of asm that name m0. Each instruction is one wait state, s_nop N has N + 1."""
    loads, bad, others, before, inside = 0, [], [], [], False
    for line in asm.split("\n"):
        if "#ASMSTART" in line or "#ASMEND" in line:
            inside = "#ASMSTART" in line
        line = line.split(";")[0].strip()
        if not line or line[0] == "." or line.endswith(":"):
            continue
        op, _, operands = line.partition(" ")
        op = op.split("\t")[0]
        operands = line[len(op):]
        if not inside and re.search(r"\bm0\b", operands):
            others.append(line)
        if re.match(r"(global|buffer)_load_.*lds|buffer_load_", op) and "lds" in line:
            loads += 1
            need, waited = scalar_registers(operands), 0
            for states, written in reversed(before):
                if waited >= 5:
                    break
                if written & need:
                    bad.append(line)
                    break
                waited += states
        vector = op.startswith("v_")
        before.append((int(operands) + 1 if op == "s_nop" else 1, scalar_registers(",".join(operands.split(",")[:2])) if vector else set()))
        del before[:-8]
    return loads, bad, others


def test_the_check_finds_what_it_looks_for():
    text = "\tv_readfirstlane_b32 s4, v1\n\t;;#ASMSTART\n\tglobal_load_lds_dwordx4 v2, s[4:5] offset:0\n\t;;#ASMEND\n"
    assert hazards(text) == (1, ["global_load_lds_dwordx4 v2, s[4:5] offset:0"], [])
    assert hazards(text.replace(";;#ASMSTART", ";;#ASMSTART\n\ts_nop 4")) == (1, [], [])
    assert hazards(text.replace(";;#ASMSTART", ";;#ASMSTART\n\ts_nop 3"))[1]
    assert hazards("\ts_mov_b32 m0, s3\n")[2]


@pytest.mark.skipif(not (os.path.exists(HIPCC) or shutil.which("hipcc")), reason="hipcc not installed")
@pytest.mark.parametrize("source", ["bpw_kv4_attention_d64.hip", "bpw_kv4_attention_d128.hip", "bpw_kv4_attention_d256.hip",
                                    "bpw_prompt_d64.hip", "bpw_attention_d64.hip"])
def test_scalar_operands_have_settled(tmp_path, source):
    spec = importlib.util.spec_from_file_location("bpw_build", os.path.join(ROOT, "bit_plane_weight_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    out = tmp_path / "kernels.s"
    source = os.path.join(CSRC, source)
    subprocess.run([HIPCC, *build.flags_for(source), "-S", "--cuda-device-only", source, "-o", str(out)], check=True, capture_output=True)
    loads, bad, others = hazards(out.read_text())
    assert loads >= 48 and not bad, bad[:5]
    assert not others, others[:5]


def unsettled_in_their_block(asm):
    """Loads to LDS with scalar operands, and those before which their own asm block does not hold five wait states: what stands there
    holds on every path to the block, also across branches."""
    loads, bad, waited, inside = 0, [], 0, False
    for line in asm.split("\n"):
        if "#ASMSTART" in line or "#ASMEND" in line:
            inside, waited = "#ASMSTART" in line, 0
        line = line.split(";")[0].strip()
        if not line or line[0] == "." or line.endswith(":"):
            continue
        op = line.split()[0]
        operands = line[len(op):]
        if re.match(r"(global|buffer)_load_", op) and "lds" in line and scalar_registers(operands):
            loads += 1
            if not inside or waited < 5:
                bad.append(line)
        waited += int(operands) + 1 if op == "s_nop" else 1
    return loads, bad


def test_the_check_of_blocks_finds_what_it_looks_for():
    load = "buffer_load_dwordx4 v2, s[4:7], 0 offen lds\n"
    good = f"\ts_nop 7\n\t;;#ASMSTART\n\ts_mov_b32 m0, s3\n\ts_nop 3\n\t{load}\t{load}\t;;#ASMEND\n"
    assert unsettled_in_their_block(good) == (2, [])
    assert len(unsettled_in_their_block(good.replace("s_nop 3", "s_nop 2"))[1]) == 1
    assert len(unsettled_in_their_block(f"\ts_nop 7\n\t{load}")[1]) == 1
    assert unsettled_in_their_block("\t;;#ASMSTART\n\tglobal_load_lds_dwordx4 v[2:3], off offset:16 nt\n\t;;#ASMEND\n") == (0, [])


@pytest.mark.skipif(not (os.path.exists(HIPCC) or shutil.which("hipcc")), reason="hipcc not installed")
@pytest.mark.parametrize("source,scalar", [("bpw_prompt_d64.hip", True), ("bpw_prompt_d128.hip", True), ("bpw_prompt_d256.hip", True),
                                           ("bpw_attention_d64.hip", True), ("bpw_attention_d128.hip", True), ("bpw_attention_d256.hip", True),
                                           ("bpw_kv4_attention_d64.hip", False), ("bpw_kv4_attention_d128.hip", False),
                                           ("bpw_kv4_attention_d256.hip", False)])
def test_scalar_operands_have_settled_on_every_path(tmp_path, source, scalar):
    """Every head size. The 4-bit attention's loads have no scalar operands."""
    spec = importlib.util.spec_from_file_location("bpw_build", os.path.join(ROOT, "bit_plane_weight_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    out = tmp_path / "kernels.s"
    source = os.path.join(CSRC, source)
    subprocess.run([HIPCC, *build.flags_for(source), "-S", "--cuda-device-only", source, "-o", str(out)], check=True, capture_output=True)
    asm = out.read_text()
    loads, bad = unsettled_in_their_block(asm)
    assert (loads >= 48 if scalar else loads == 0) and not bad, (loads, bad[:5])
    loads, bad, others = hazards(asm)
    assert loads >= 48 and not bad and not others, (loads, bad[:5], others[:5])
