// The 16-byte pieces in which values of a row come where the row begins
// anywhere: plain arithmetic, of the host too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SGEMM_ROW_PIECES __host__ __device__ __forceinline__
#else
#define SGEMM_ROW_PIECES inline
#endif

namespace sgemm_gb300 {

// Bytes [lo, hi) of the 16 from `from` on.
struct RowPiece {
    uintptr_t from;
    int lo, hi;
    SGEMM_ROW_PIECES bool some() const { return lo < hi; }
    SGEMM_ROW_PIECES bool whole() const { return lo == 0 && hi == 16; }
};

// Piece q of those that hold the `bytes` from `at` on, values that lie in
// [row, row_end): of the 16 bytes what is in there, as what is before and behind
// may not be read; nothing where the `bytes` end before the piece.
SGEMM_ROW_PIECES RowPiece row_piece(uintptr_t row, uintptr_t row_end, uintptr_t at, int bytes, int q)
{
    RowPiece p{(at & ~uintptr_t(15)) + 16 * (uintptr_t)q, 0, 16};
    if (p.from < row) p.lo = (int)(row - p.from);
    if (p.from >= at + bytes) p.hi = 0;
    else if (p.from + 16 > row_end) p.hi = (int)(row_end - p.from);
    return p;
}

}  // namespace sgemm_gb300
