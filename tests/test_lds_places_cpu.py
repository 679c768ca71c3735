"""Where the backward pass of the head norm has its arrays in LDS: 16-byte accesses
are 16-byte aligned for every head size."""
import os
import shutil
import subprocess

import pytest

from collective_communication_ring_amd import build

SOURCE = r"""
#include <cstdio>
#include "ar_heads.h"
int main()
{
    for (uint32_t dim = 1; dim <= ar::kHeadMaxDim; ++dim)
        for (uint32_t angles : {0u, 1u, 5u, 512u}) {  // of a wave
            const ar::HeadBackPlaces p = ar::head_back_places(dim, 256, 4, angles);
            if (p.sums % 16 || p.sums < 8 * dim || p.angles % 8 || p.angles < p.sums + 256 * 16 * 4 ||
                p.bytes < p.angles + 4 * angles * 8 || p.bytes < 4 * dim * 4) {
                std::printf("%u %u: %u %u %u\n", dim, angles, p.sums, p.angles, p.bytes);
                return 1;
            }
        }
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"),
                    reason="g++ or HIP's headers are not installed")
def test_backward_pass_of_the_head_norm(tmp_path):
    (tmp_path / "places.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-w", "-I", "/opt/rocm/include", "-I",
                    os.path.join(build.ROOT, "include"), "-I", build.CSRC, str(tmp_path / "places.cpp"),
                    "-o", str(tmp_path / "places")], check=True)
    r = subprocess.run([str(tmp_path / "places")], stdout=subprocess.PIPE, text=True)
    assert r.returncode == 0, r.stdout
