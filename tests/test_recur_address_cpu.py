"""Where the recurrence's lanes read and write: the kernels' own address
arithmetic compiled for the host."""
import os
import subprocess

import pytest

from laplace_matvec_amd import build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "lx_recur.h"

// Every lane of every wave that has a row: the address of its row j, clamped
// to the last row as its loads are, against that row's address.
template <class T, int V, int L>
void lanes(int64_t n, int64_t width, int64_t ld, long& bad)
{
    using Lay = lx::RecurLayout<V, L>;
    char* const base = (char*)((uintptr_t)1 << 60);
    const int64_t pitch = lx::recur_pitch(n, width, ld);
    for (int wave = 0; wave < Lay::kThreads / lx::kWave; ++wave) {
        const int64_t wave_row = (int64_t)wave * (lx::kWave / Lay::kLanes) * L;
        if (wave_row >= n) break;
        for (int lane = 0; lane < lx::kWave; ++lane) {
            const int lane_row = lane / Lay::kLanes * L;
            const int64_t end = lane % Lay::kLanes * V + V, col = (end < width ? end : width) - V;
            const lx::RowAt<T, V> at(base, pitch, wave_row, lane_row, (int)(col > 0 ? col : 0));
            const int64_t last = n - 1 - wave_row - lane_row;
            for (int64_t j = 0; j < L; ++j) {
                const char* p = (const char*)at.any_row(j < last ? j : last);
                const int64_t row = wave_row + lane_row + (j < last ? j : last);
                bad += row < 0 || row >= n || p != base + (row * pitch + (col > 0 ? col : 0)) * (int64_t)sizeof(T);
            }
        }
    }
}

int main(int argc, char** argv)
{
    const int64_t n = atoll(argv[1]), ld = atoll(argv[2]), width = 64;
    long bad = 0;
    lanes<float, 4, 16>(n, width, ld, bad);
    lanes<float, 4, 8>(n, width, ld, bad);
    lanes<float, 4, 4>(n, width, ld, bad);
    lanes<float, 1, 16>(n, width, ld, bad);
    lanes<uint16_t, 4, 16>(n, width, ld, bad);
    lanes<uint16_t, 4, 4>(n, width, ld, bad);
    printf("%ld\n", bad);
    return bad != 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("lanes")
    src, exe = at / "lanes.hip", at / "lanes"
    src.write_text(PROGRAM)
    subprocess.run([build.HIPCC, "--offload-host-only", "-O1", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC,
                    str(src), "-o", str(exe)], check=True, capture_output=True, timeout=300)
    return str(exe)


# one row may come with any pitch, more with the largest there is
@pytest.mark.parametrize("n,ld", [(1, 64), (1, 23000000), (1, 1 << 27), (1, 1 << 28), (1, 1 << 30), (1, 1 << 40),
                                  (2, 64), (2, 1 << 24), (3, 1 << 24), (17, 1 << 24), (49, 1 << 24), (255, 1 << 24),
                                  (256, 1 << 24)])
def test_lanes_stay_within_the_rows(program, n, ld):
    r = subprocess.run([program, str(n), str(ld)], capture_output=True, text=True, timeout=60, env=dict(os.environ))
    assert r.returncode == 0 and r.stdout == "0\n", r.stdout + r.stderr
