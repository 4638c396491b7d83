"""Where the kernels read, over every length, as the kernels compute it: on the CPU."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_ragged_grouped_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "cake_gg_int8_index.h"
using namespace cakegg;
int main()
{
    for (int K = 16; K < 1 << 17; K += K < 4096 ? 16 : 4096 - 16 * 3) {
        long long read = 0;
        for (int s = 0; s <= (K + 63) / 64 + 8; ++s)        // (steps past the row's too: they are asked for ahead)
            for (int lane = 0; lane < 32; ++lane) {
                const int at = i8_warps_token(s, lane, K);
                if (at < 0 || at % 16 != 0 || at + 16 > K) return std::printf("K %d step %d lane %d reads %d\n", K, s, lane, at), 1;
                if (i8_warps_in(s, lane, K)) {
                    if (at != s * 64 + i8_warps_place(lane)) return std::printf("K %d step %d lane %d: %d\n", K, s, lane, at), 1;
                    read += 16;
                }
            }
        if (read != 8ll * K) return std::printf("K %d: %lld bytes by 8 groups of lanes\n", K, read), 1;
    }
    return 0;
}
"""


def test_lanes_of_the_warp_path_stay_in_their_rows(tmp_path):
    """Every lane's 16 bytes lie in the row, also of rows shorter than a step; together they are the row."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    src, exe = tmp_path / "index.cpp", tmp_path / "index"
    src.write_text(PROGRAM)
    built = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)],
                           capture_output=True, text=True, timeout=120)
    assert built.returncode == 0, built.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout
