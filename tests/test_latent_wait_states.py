"""The latent attention kernels keep their sums in accumulation registers through
matrix instructions that the compiler does not see as such, so nothing but the
source keeps other instructions from reading a sum before it is there.  This
walks the assembly of the kernels, built here with the library's own flags,
along every path from such an instruction."""

import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = "rts_latent.hip"
# A result of the longest matrix instruction may be touched 19 wait states
# later; an instruction is one, s_nop k is k + 1.
NEED = 19


def build_script():
    spec = importlib.util.spec_from_file_location("_rts_build", os.path.join(ROOT, "row_top_select_amd", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    return b


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    b = build_script()
    out = str(tmp_path_factory.mktemp("asm") / "latent.s")
    cmd = [b.HIPCC, *b.COMMON, *b.EXTRA[SRC], "-S", "--offload-device-only", os.path.join(b.CSRC, SRC), "-o", out]
    subprocess.run(cmd, check=True, capture_output=True)
    found = re.findall(r"^(\w*latent_attend_kernel\w*):(.*?)\.end_amdhsa_kernel", open(out).read(), flags=re.M | re.S)
    return {name: parse(body) for name, body in found}


def parse(body):
    """[(operation, operands)] and {label: index}."""
    code, labels = [], {}
    for line in body.splitlines():
        line = line.split(";")[0].split("//")[0].strip()
        m = re.match(r"^(\.\w+):$", line)
        if m:
            labels[m[1]] = len(code)
        elif line and not line.startswith(".") and not line.endswith(":"):
            op, *rest = line.replace(",", " ").split()
            code.append((op, rest))
    return code, labels


def accumulators(token):
    m = re.match(r"^-?\|?a\[(\d+):(\d+)\]", token)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.match(r"^-?\|?a(\d+)\b", token)
    return {int(m[1])} if m else set()


def too_early(code, labels, start):
    """The first instruction that touches the result of code[start] before it is there, on any path."""
    regs = accumulators(code[start][1][0])
    best, todo = {}, [(start + 1, 0)]
    while todo:
        i, waited = todo.pop()
        if waited >= NEED or i >= len(code) or best.get(i, NEED) <= waited:
            continue
        best[i] = waited
        op, rest = code[i]
        if op == "s_endpgm":
            continue
        touched = set().union(*(accumulators(t) for t in rest)) & regs
        # The next product of the same sum is the one reader that may come at once.
        if touched and not (op.startswith("v_mfma") and accumulators(rest[0]) == regs):
            return i
        if touched:
            continue  # checked from there
        waited += int(rest[0]) + 1 if op == "s_nop" else 1
        if op.startswith("s_cbranch") or op == "s_branch":
            todo.append((labels[rest[0]], waited))
            if op == "s_branch":
                continue
        todo.append((i + 1, waited))
    return None


def test_sums_are_waited_for(kernels):
    assert len(kernels) == 12
    for name, (code, labels) in kernels.items():
        products = [i for i, (op, rest) in enumerate(code) if op.startswith("v_mfma") and accumulators(rest[0])]
        assert products, name
        for i in products:
            at = too_early(code, labels, i)
            assert at is None, f"{name}: {code[i]} then {code[at]} after {at - i} instructions"
            # s_nop 1 in front: two wait states after whatever wrote an operand
            assert code[i - 1] == ("s_nop", ["1"]), name


def test_the_walk_finds_an_early_read():
    code, labels = parse("""
        s_nop 1
        v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]
        s_cbranch_scc1 .L1
        s_nop 15
        s_nop 7
        v_accvgpr_read_b32 v0, a3
    .L1:
        v_mov_b32 v1, v2
        v_accvgpr_read_b32 v0, a15
        s_endpgm
    """)
    assert too_early(code, labels, 1) == 7
    ok, lab = parse("""
        v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]
        v_accvgpr_read_b32 v0, a16
        s_nop 15
        s_nop 7
        v_accvgpr_read_b32 v0, a3
    """)
    assert too_early(ok, lab, 0) is None
