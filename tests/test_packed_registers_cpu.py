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


def test_the_compiler_gives_the_kernels_what_the_roles_share(tmp_path):
    # a kernel with fewer registers at launch is refused by every call: seen here, before that
    import shutil
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    import importlib.util
    spec = importlib.util.spec_from_file_location(
        "_sa_build", os.path.join(ROOT, "head_heterogeneous_block_gb300", "_build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    r = subprocess.run([nvcc, *build.ARCH, "-O3", "-std=c++17", f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-Xptxas", "-v",
                        "-c", SOURCE, "-o", str(tmp_path / "packed.o")], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    used = [int(n) for n in re.findall(r"entry function '\S*packed_attention_kernel\S*'.*?Used (\d+) registers",
                                       r.stdout + r.stderr, re.S)]
    text = open(SOURCE).read()
    regs = {name: int(n) for name, n in re.findall(r"\b(k\w+Regs) = (\d+)", text)}
    threads = {name: int(n) for name, n in re.findall(r"constexpr int (k\w+Threads) = (\d+);", text)}
    need = (128 * regs["kControlRegs"] + threads["kSoftmaxThreads"] * regs["kSoftmaxRegs"] +
            threads["kOutThreads"] * regs["kOutRegs"])
    all_threads = 128 + threads["kSoftmaxThreads"] + threads["kOutThreads"]
    assert len(used) == 8 and all(all_threads * (-(-n // 8) * 8) >= need for n in used), (used, need)
