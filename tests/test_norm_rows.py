"""The index arithmetic of the layer norm's rows (csrc/norm_rows.h), walked on the host: every piece that a kernel loads
whole lies inside the tensor, and the pieces of a row cover its columns once."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fft_long_convolution_causal_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "norm_rows.h"
using namespace fftc::ln;

// a row's pieces as threads of TPR hold them, E each; V elements are 16 bytes
template <int V, int TPR, int E, bool OFF>
int walk(int64_t rows, int C) {
    const int64_t size = rows * C;
    for (int64_t r = 0; r < rows; ++r) {
        std::vector<int> seen(C, 0);
        const int end = to_end(r, rows, C);
        for (int lane = 0; lane < TPR; ++lane) {
            const Pieces<V, TPR, OFF> p{lane, offset<V, OFF>(r, C), C};
            for (int i = 0; i < E; ++i) {
                if (!p.any(i)) continue;
                const int64_t at = r * C + p.first(i);
                if (at % V) return printf("rows %d C %d V %d: row %d lane %d off the boundary\n", (int)rows, C, V, (int)r, lane);
                if (p.whole(i, end) && (at < 0 || at + V > size))
                    return printf("rows %d C %d V %d: row %d lane %d loads elements %d to %d of %d\n", (int)rows, C, V, (int)r,
                                  lane, (int)at, (int)at + V, (int)size);
                bool all = true;
                for (int c = p.first(i); c < p.first(i) + V; ++c) {
                    all = all && p.has(c);
                    if (p.has(c)) ++seen[c];
                }
                if (all != p.inside(i)) return printf("rows %d C %d V %d: row %d inside\n", (int)rows, C, V, (int)r);
            }
        }
        for (int c = 0; c < C; ++c)
            if (seen[c] != 1) return printf("rows %d C %d V %d: row %d column %d held %d times\n", (int)rows, C, V, (int)r, c, seen[c]);
    }
    return 0;
}
template <int V>
int all() {
    const int64_t some[] = {1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 17, 1000};
    for (int64_t rows : some) {
        for (int C = 1; C <= 8 * V - V + 1; ++C) {
            if (C % V && walk<V, 8, 1, true>(rows, C)) return 1;
            if (C % V == 0 && walk<V, 8, 1, false>(rows, C)) return 1;
        }
        for (int C = 8 * V - V + 2; C <= 16 * V - V + 1; ++C)
            if (C % V && walk<V, 8, 2, true>(rows, C)) return 1;
        if (rows < 20 && (walk<V, 128, 2, true>(rows, 128 * V + 3) || walk<V, 512, 1, true>(rows, 512 * V - 7))) return 1;
    }
    // far from the end of a long tensor, and at it
    const int64_t rows = int64_t(1) << 31;
    if (to_end(0, rows, 16383) != 1 << 30 || to_end(rows - 1, rows, 16383) != 16383 || to_end(rows - 2, rows, 1) != 2)
        return printf("to_end\n");
    return 0;
}
int main() { return all<8>() || all<4>() ? 1 : 0; }
"""


def test_whole_pieces_lie_inside_the_tensor(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    source, program = tmp_path / "rows.cpp", tmp_path / "rows"
    source.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, str(source), "-o", str(program)], check=True)
    r = subprocess.run([str(program)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
