"""csrc/resident.h on the host: a kernel's count of resident blocks is its own."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "resident.h"
#include <cstdio>

// two kernels of one type, as the instances of a template on their loads are
template <bool NT> void kernel(int) {}

static int asked;
template <bool NT> int64_t blocks(int gpu, int64_t n) {
    return sq::once_per_gpu<kernel<NT>>(gpu, [&] { ++asked; return n; });
}

int main() {
    if (blocks<true>(0, 512) != 512 || blocks<false>(0, 256) != 256) return 1;   // its own value
    if (blocks<true>(0, 1) != 512 || blocks<false>(0, 1) != 256 || asked != 2) return 2;  // asked once
    if (blocks<true>(1, 128) != 128 || blocks<true>(0, 1) != 512) return 3;      // and per GPU
    if (blocks<true>(64, 7) != 7 || blocks<true>(64, 9) != 9 || blocks<true>(-1, 5) != 5) return 4;
    return 0;
}
"""


def test_counts_belong_to_a_kernel_and_a_gpu(tmp_path):
    src, exe = tmp_path / "resident.cpp", tmp_path / "resident"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "w8a8_post_quantization_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", inc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
