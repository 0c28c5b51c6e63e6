"""The generated code of the 8-bit product: the compiler does not see the matrix
instructions in their inline assembly, so that nothing but the source's own waits
keeps an accumulator's readers away from them. Along every path of the compiled
kernels, no accumulator is moved between a matrix instruction and the wait that
settles it, and no value goes through scratch memory."""
import os
import re
import subprocess

import pytest

from quantized_sgd_amd import build


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("code") / "int8.s")
    source = os.path.join(build.HERE, "csrc", "int8_api.hip")
    subprocess.run(build.compile_command(source, out, ("--cuda-device-only", "-S")), check=True, capture_output=True)
    with open(out) as f:
        return f.read()


def kernels(text):
    """{name: instructions and labels} of the product's tile kernels."""
    found, name = {}, None
    for line in text.splitlines():
        m = re.match(r"(_ZN\S*matmul\w*kernel\S*):", line)
        if m:
            name = m.group(1)
            found[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name:
            found[name].append(line.split(";")[0].strip())
    return found


def unsettled(code):
    """Instructions that move accumulators where a matrix instruction may still be writing them."""
    labels = {line[:-1]: i for i, line in enumerate(code) if line.startswith(".LBB") and line.endswith(":")}
    bad, seen, work = [], set(), [(0, False)]
    while work:
        i, pending = work.pop()
        while i < len(code) and (i, pending) not in seen:
            seen.add((i, pending))
            line = code[i]
            if line.startswith("v_mfma"):
                pending = True
            elif line.startswith("s_nop 15"):
                pending = False
            elif pending and (line.startswith("v_accvgpr") or re.match(r"(scratch|global|buffer|ds)_\S+.*\ba(\d|\[)", line)):
                bad.append(line)
            if line.startswith("s_endpgm"):
                break
            jump = re.match(r"s_c?branch\S*\s+(\.LBB\S+)", line)
            if jump:
                work.append((labels[jump.group(1)], pending))
                if line.startswith("s_branch"):
                    break
            i += 1
    return bad


def test_accumulators_are_settled_before_they_are_read(assembly):
    code = kernels(assembly)
    assert len(code) == 15  # three tiles by three types, two tiles by three types in pairs
    for name, lines in code.items():
        assert sum(line.startswith("v_mfma") for line in lines) > 0, name
        assert unsettled(lines) == [], name


def test_the_check_sees_an_early_read():
    code = ["v_mfma_i32_16x16x64_i8 a[0:3], v[0:3], v[4:7], a[0:3]", "s_cbranch_scc1 .LBB0_2", "s_nop 15", ".LBB0_2:",
            "v_accvgpr_read_b32 v0, a0", "s_endpgm"]
    assert unsettled(code) == ["v_accvgpr_read_b32 v0, a0"]
    assert unsettled(code[:1] + code[2:]) == []


def test_no_scratch_memory(assembly):
    sizes = re.findall(r"\.name:\s+(_ZN\S*matmul\w*kernel\S*)\s+\.private_segment_fixed_size:\s+(\d+)", assembly)
    assert len(sizes) == 15
    assert [name for name, size in sizes if int(size)] == []
