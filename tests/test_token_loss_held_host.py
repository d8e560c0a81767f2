"""Rows that a workgroup holds between its sums and its gradients: the device
code's own indices, compiled for the CPU (support/held_rows_host.cpp) and run for
every workgroup size up to its capacity, both types, several places in a cache
line.  CPU only."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fsdp_sharded_optimizer_flat_amd", "csrc")
SUPPORT = os.path.join(ROOT, "tests", "support")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def held_chunks(name):
    return int(re.search(r"constexpr int kHeld = (\d+);", source(name)).group(1))


def test_held_rows_are_summed_and_written_once(tmp_path):
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    clang = os.path.join(rocm, "llvm", "bin", "clang++")
    if not os.path.exists(clang):
        clang = shutil.which("clang++")
    if not clang:
        pytest.skip("needs clang (vector types and bf16 on the host)")
    # the workgroup sizes that the program goes through are the kernels'
    for name, sizes in (("logprob_kernels.hip", (64, 256, 512, 1024)), ("distill_kernels.hip", (64, 192, 448, 960))):
        held = source(name)[source(name).index("int held_threads("):]
        assert tuple(int(n) for n in re.findall(r"most <= (\d+) \* kHeld", held)) == sizes, name
    exe = str(tmp_path / "held_rows")
    subprocess.run([clang, "-std=c++17", "-O1", f"-DLOGPROB_HELD={held_chunks('logprob_kernels.hip')}",
                    f"-DDISTILL_HELD={held_chunks('distill_kernels.hip')}",
                    "-I", os.path.join(SUPPORT, "host_device"), "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(SUPPORT, "held_rows_host.cpp"), "-o", exe], check=True, timeout=300)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    lines = res.stdout.splitlines()
    assert sum("cases, 0 wrong" in line for line in lines) == 16 and res.returncode == 0, res.stdout[-3000:]
