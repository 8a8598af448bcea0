"""Which bytes of a joined matrix are read where TMA cannot address it
(no GPU): the arithmetic of csrc/row_pieces.cuh, compiled for the host, byte by
byte. All of a chunk's values come, in the pieces that its buffer has room for,
and nothing outside the row: what lies between a row's last value and its
leading dimension belongs to others."""

import itertools
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# For each line "row row_end at bytes pieces size": the bytes read of the row's surroundings, by offset from `row`.
PROGRAM = r"""
#include "row_pieces.cuh"
#include <cstdio>
int main()
{
    unsigned long long row, end, at;
    int bytes, pieces, size;
    while (std::scanf("%llu %llu %llu %d %d %d", &row, &end, &at, &bytes, &pieces, &size) == 6) {
        for (int q = 0; q < pieces; ++q) {
            const sgemm_gb300::RowPiece p = sgemm_gb300::row_piece(row, end, at, bytes, q);
            if (!p.some()) continue;
            if (p.lo % size || p.hi % size) std::printf("x ");
            if (p.whole() != (p.hi - p.lo == 16)) std::printf("x ");
            for (int e = p.lo; e < p.hi; ++e) std::printf("%lld ", (long long)(p.from + e) - (long long)row);
        }
        std::printf("\n");
    }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    compiler = shutil.which("g++") or shutil.which("c++")
    assert compiler, "a C++ compiler"
    at = tmp_path_factory.mktemp("row_pieces")
    (at / "main.cpp").write_text(PROGRAM)
    subprocess.run([compiler, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "dense_fp32_matrix_07_gb300", "csrc"), str(at / "main.cpp"),
                    "-o", str(at / "main")], check=True)
    return str(at / "main")


@pytest.mark.parametrize("size,pieces", [(4, 9), (2, 5)], ids=["f32", "bf16"])
def test_pieces_hold_the_chunk_and_stay_in_the_row(program, size, pieces):
    cases = []
    for shift, cols in itertools.product(range(16 // size), (1, 2, 3, 7, 31, 32, 33, 61, 63, 64, 65, 96, 97, 131)):
        row = (1 << 40) + 32 + shift * size
        for n in range(0, cols, 32):
            cases.append((row, row + cols * size, row + n * size, min(cols - n, 32) * size, pieces, size))
    out = subprocess.run([program], input="\n".join(" ".join(map(str, c)) for c in cases), text=True, capture_output=True, check=True).stdout
    lines = out.splitlines()
    assert len(lines) == len(cases)
    for (row, end, at, bytes_, *_), line in zip(cases, lines):
        read = [int(x) for x in line.split()]
        assert len(set(read)) == len(read)
        assert min(read) >= 0 and max(read) < end - row, "outside the row"
        assert set(range(at - row, at - row + bytes_)) <= set(read), "a value is missing"
