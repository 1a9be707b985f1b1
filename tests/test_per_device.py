"""What moe_init measures of a device stays that device's: the table itself with
a stand-in for the current device, and that every launch plan goes by it."""
import os
import re
import shutil
import subprocess

import pytest

from helpers import ROOT

CSRC = os.path.join(ROOT, "grouped_gemm_top_gb300", "csrc")

PROGRAM = r"""
#include <initializer_list>
#include "per_device.cuh"
static int current = 0;
extern "C" cudaError_t cudaGetDevice(int* d) { return *d = current, current == 99 ? cudaErrorNoDevice : cudaSuccess; }
struct Most { int n[3]; };
static moe::PerDevice<Most> most;
int main() {
    for (current = 0; current < 64; ++current)
        if (most.here().n[1] != 0) return 1;
    current = 0, most.here().n[1] = 76;
    current = 5, most.here().n[1] = 12;
    current = 0;
    if (most.here().n[1] != 76) return 2;
    current = 5;
    if (most.here().n[1] != 12) return 3;
    for (int dev : {99, -1, 64}) {      // none: zeros, and nothing that a write leaves there
        current = dev;
        if (most.here().n[1] != 0) return 4;
        most.here().n[1] = 7;
        if (most.here().n[1] != 0) return 5;
    }
    current = 0;
    return most.here().n[1] == 76 && most.here().n[0] == 0 ? 0 : 6;
}
"""


def test_table(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cxx = shutil.which("g++")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if cxx is None or not os.path.exists(os.path.join(include, "cuda_runtime_api.h")):
        pytest.skip("no C++ compiler or no CUDA headers")
    (tmp_path / "t.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "t")
    r = subprocess.run([cxx, "-std=c++17", "-I", CSRC, "-I", include, "-x", "c++", str(tmp_path / "t.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([exe]).returncode == 0


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith(".cu")))
def test_no_table_of_one_device_alone(name):
    with open(os.path.join(CSRC, name)) as f:
        src = f.read()
    if "cudaOccupancyMaxActiveClusters" in src:
        assert re.search(r"static PerDevice<\w+> g_\w*clusters;", src), name
    assert not re.search(r"^static int g_\w*clusters\b", src, re.M), name
