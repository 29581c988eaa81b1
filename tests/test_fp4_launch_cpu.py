"""The host side of the FP4 decode's launch, over a stand-in for the CUDA runtime
(fake_cudart.cu): no GPU."""
import os
import re
import shutil
import subprocess

import pytest

from mla_decode_attention_paged_gb300 import build as mla_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
REGISTERS = 96  # of a thread: 640 threads x 96 are what the 32-row kernel's roles share out


@pytest.fixture(scope="module")
def launch(tmp_path_factory):
    """launch(rows, q_len, registers) -> (compiled kernels, what the launches did)."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    mla_build.build()
    source = os.path.join(mla_build.CSRC, "decode_fp4.cu")
    obj = os.path.join(mla_build.BUILD_DIR, "decode_fp4.cu.o")
    if not os.path.exists(obj) or any(os.path.getmtime(p) > os.path.getmtime(obj) for p in mla_build._deps()):
        os.makedirs(mla_build.BUILD_DIR, exist_ok=True)
        mla_build._compile(source, False)
    at = tmp_path_factory.mktemp("fake_cudart")
    call, rest, exe = str(at / "call.o"), str(at / "rest.o"), str(at / "fake_cudart")
    fake = os.path.join(ROOT, "tests", "fake_cudart.cpp")
    for cmd in ([mla_build.nvcc(), "-x", "cu", "-std=c++17", "--expt-relaxed-constexpr", *mla_build.ARCH, "-I", mla_build.CSRC,
                 "-c", fake, "-o", call],
                ["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(CUDA, "include"), "-c", fake, "-o", rest],
                ["g++", call, rest, obj, "-o", exe]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr

    def run(rows, q_len, registers):
        r = subprocess.run([exe, str(rows), str(q_len), str(registers)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stdout + r.stderr
        lines = [line.split(" ", 1) for line in r.stdout.splitlines()]
        form = lambda name: tuple(int(v) for v in re.search(r"decode_fp4_kernelILi(\d+)ELb([01])E", name).groups())
        kernels = sorted(form(v) for k, v in lines if k == "kernel")
        return kernels, [form(v) if k == "launched" else k for k, v in lines if k != "kernel"]

    return run


@pytest.mark.parametrize("rows,q_len", [(16, 1), (32, 1), (32, 2)])
def test_launches_its_form(launch, rows, q_len):
    assert launch(rows, q_len, REGISTERS)[1] == [(rows, int(q_len > 1))] * 2


@pytest.mark.parametrize("q_len", [1, 2])
@pytest.mark.parametrize("registers", [64, 80, 88, 104])
def test_other_register_counts_are_not_launched(launch, q_len, registers):
    """The 32-row kernel's roles exchange registers: with fewer at the launch than they
    are meant to share, a warp would wait without end for its own."""
    assert launch(32, q_len, registers)[1] == ["refused"] * 2


@pytest.mark.parametrize("registers", [89, 95, 96])
def test_registers_are_given_out_by_eights(launch, registers):
    assert launch(32, 1, registers)[1] == [(32, 0)] * 2


def test_only_forms_that_a_call_reaches(launch):
    """16 rows are one token's (heads come by 16 or by 32): no causal form of them."""
    assert launch(16, 1, REGISTERS)[0] == [(16, 0), (32, 0), (32, 1)]
