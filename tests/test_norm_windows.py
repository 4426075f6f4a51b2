"""The windows in which the norm's rings copy rows stay inside the matrix and cover it."""
import subprocess

from conftest import ROOT

PROGRAM = r"""
#include <stdio.h>
#include "mbtile_rows.h"
int main() {
    long checked = 0;
    for (int es = 2; es <= 4; es += 2)
        for (int64_t N = 1; N <= 40; ++N)
            for (int64_t ld = N; ld <= N + 17; ++ld)
                for (int64_t M = 1; M <= 40; ++M) {
                    const int64_t pitch = ld * es, bytes = N * es, end = (M - 1) * pitch + bytes;
                    const bool phased = M > 1 && pitch % 16 != 0;
                    const int64_t tail = mbt::first_tail_row(M, bytes, pitch);
                    for (int64_t row = 0; row < M; ++row) {
                        const mbt::RowWindow w = mbt::row_window(row, tail, (int)bytes, pitch, phased);
                        const int64_t first = row * pitch, last = first + bytes;
                        // what is not copied is the row's part of the matrix's last chunk, taken from there
                        const bool whole = w.start + w.bytes >= last;
                        if (w.start < 0 || w.start % 16 || w.bytes % 16 || w.bytes < 0 || w.start + w.bytes > end ||
                            w.start + w.lead != first || w.lead > 15 || (row < tail) > whole ||
                            (!whole && (w.start + w.bytes != (last & ~15ll) || last <= (end & ~15ll)))) {
                            printf("es %d N %lld ld %lld M %lld row %lld\n", es, (long long)N, (long long)ld,
                                   (long long)M, (long long)row);
                            return 1;
                        }
                        ++checked;
                    }
                }
    printf("%ld\n", checked);
    return 0;
}
"""


def test_windows_stay_inside_the_matrix(tmp_path):
    src, exe = tmp_path / "w.cpp", tmp_path / "w"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", f"{ROOT}/mbarrier_async_tile_gb300/csrc", str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert got.returncode == 0, got.stdout
    assert int(got.stdout) == 2 * 40 * 18 * sum(range(1, 41))
