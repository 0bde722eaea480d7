"""The loads that are written out by hand, as test_direct_loads_cpu looks at them, in the kernels of token log
probabilities and distillation, which are made of the same products."""

import os
import re
import subprocess

import pytest

import test_direct_loads_cpu as direct
from test_learned_neural_amd import build


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """Instructions of each kernel, in order; None where a branch may arrive."""
    found = {}
    for source in ("k_logprobs.hip", "k_distill.hip"):
        out = tmp_path_factory.mktemp("asm") / "k.s"
        flags = [f for f in build.FLAGS if f not in ("-fPIC", "-Wall")]
        subprocess.run([build.hipcc(), *flags, "-S", "--cuda-device-only", os.path.join(build.CSRC, source), "-o",
                        str(out)], check=True, capture_output=True)
        name = None
        for line in out.read_text().splitlines():
            label = re.match(r"(\S+):", line)
            if label:
                if label[1].startswith("_Z"):
                    name = source, label[1]
                    found[name] = []
                elif name:
                    found[name].append(None)
                continue
            text = line.split(";")[0].strip()
            if name and text and not text.startswith("."):
                found[name].append(text)
    return {k: v for k, v in found.items() if any(i and direct.LOAD.match(i) for i in v)}


def test_loads(code):
    direct.test_every_load_sets_m0_and_puts_it_back(code)
    direct.test_no_load_reads_a_register_that_a_vector_instruction_just_wrote(code)


def test_no_kernel_keeps_registers_in_memory(code):
    """A load in flight writes LDS, not registers: a spill between it and its wait would only be slow, but is not there."""
    for name, lines in code.items():
        assert not any(i and re.match(r"scratch_(load|store)", i) for i in lines), name
