"""The packed attention's registers by role, from its source and what the compiler
gives its kernels (no GPU)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "head_heterogeneous_block_gb300", "csrc", "packed.cu")


def test_a_warpgroup_sets_its_registers_with_one_instruction():
    # one for warps 0 to 3, one for the softmax groups, one for the output group
    text = open(SOURCE).read()
    given = re.findall(r"registers_(dec|inc)<(\w+)>\(\)", text)
    assert sorted(given) == [("dec", "kControlRegs"), ("dec", "kSoftmaxRegs"), ("inc", "kOutRegs")]
