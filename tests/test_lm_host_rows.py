"""The rows that each thread of the norm's kernels visits, counted on the CPU from
the header that the kernels take them from."""
import subprocess

from scan_linear_recurrences_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "mgs_rows.h"
int main() {
    for (int tpr : {8, 16, 32, 64, 160, 512})
        for (int64_t rows = 1; rows < 70; ++rows)
            for (unsigned blocks : {1u, 2u, 3u, 8u}) {
                const unsigned threads = tpr > 32 ? tpr : 128;
                std::vector<int> seen(rows, 0);
                for (unsigned b = 0; b < blocks; ++b) {
                    int rounds = -1;
                    for (unsigned t = 0; t < threads; ++t) {
                        mgs::RowWalk at(b, blocks, t, threads, tpr);
                        int n = 0;
                        for (; at.more(rows); at.next(), ++n)
                            if (at.row < rows) ++seen[at.row];
                        if (t == 0) rounds = n;
                        if (n != rounds) return printf("tpr %d rows %d blocks %u block %u thread %u: %d rounds, not %d\n", tpr, int(rows), blocks, b, t, n, rounds), 1;
                    }
                }
                for (int64_t r = 0; r < rows; ++r)
                    if (seen[r] != tpr) return printf("tpr %d rows %d blocks %u: row %d visited by %d threads\n", tpr, int(rows), blocks, int(r), seen[r]), 1;
            }
    return 0;
}
"""


def test_threads_of_a_block_go_round_together(tmp_path):
    # they shuffle with all lanes of their warp: one that left a round early would be missing in the next
    src, exe = tmp_path / "rows.cpp", tmp_path / "rows"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
