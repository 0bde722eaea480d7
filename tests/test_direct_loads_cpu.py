"""The loads that cross entropy writes out by hand (memory straight to LDS), in the source and in the assembly
that the build's own flags give: each has its LDS address in m0 and puts back what was there (the compiler
takes m0 for its own), and no register of its buffer was written by a vector instruction less than five wait
states before (the compiler, which keeps that distance for its own loads, does not look inside)."""

import os
import re
import subprocess

import pytest

from test_learned_neural_amd import build

SOURCE = os.path.join(build.CSRC, "k_xent.hip")
LOAD = re.compile(r"buffer_load_dwordx4 v\d+, s\[(\d+):(\d+)\], 0 offen lds$")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Instructions of each kernel, in order; None where a branch may arrive."""
    out = tmp_path_factory.mktemp("asm") / "k_xent.s"
    flags = [f for f in build.FLAGS if f not in ("-fPIC", "-Wall")]
    subprocess.run([build.hipcc(), *flags, "-S", "--cuda-device-only", SOURCE, "-o", str(out)], check=True,
                   capture_output=True)
    found, name = {}, None
    for line in out.read_text().splitlines():
        label = re.match(r"(\S+):", line)
        if label:
            if label[1].startswith("_Z"):
                name = label[1]
                found[name] = []
            elif name:
                found[name].append(None)
            continue
        text = line.split(";")[0].strip()
        if name and text and not text.startswith("."):
            found[name].append(text)
    return {k: v for k, v in found.items() if any(i and LOAD.match(i) for i in v)}


def test_every_load_sets_m0_and_puts_it_back(kernels):
    assert len(kernels) >= 16
    for name, code in kernels.items():
        loads = [k for k, i in enumerate(code) if i and LOAD.match(i)]
        for k in loads:
            kept = re.match(r"s_mov_b32 (s\d+), m0$", code[k - 3] or "")
            assert kept, (name, code[k - 3:k + 2])
            address = re.match(r"s_mov_b32 m0, (s\d+)$", code[k - 2] or "")
            assert address and address[1] != kept[1] and code[k - 1] == "s_nop 0", (name, code[k - 3:k + 2])
            assert code[k + 1] == f"s_mov_b32 m0, {kept[1]}", (name, code[k - 3:k + 2])


def test_no_load_reads_a_register_that_a_vector_instruction_just_wrote(kernels):
    for name, code in kernels.items():
        for k, i in enumerate(code):
            m = i and LOAD.match(i)
            if not m:
                continue
            own, waits = range(int(m[1]), int(m[2]) + 1), 0
            for j in range(k - 1, -1, -1):
                if waits >= 5:
                    break
                t = code[j]
                if t is None:
                    continue
                nop = re.match(r"s_nop (\d+)", t)
                if t.startswith("v_"):
                    first = t.split(None, 1)[1].split(",")[0]
                    wrote = re.match(r"s(\d+)$|s\[(\d+):(\d+)\]$", first)
                    if wrote:
                        a, b = int(wrote[1] or wrote[2]), int(wrote[1] or wrote[3])
                        assert b < own[0] or a > own[-1], (name, t, i, waits)
                waits += int(nop[1]) + 1 if nop else 1
