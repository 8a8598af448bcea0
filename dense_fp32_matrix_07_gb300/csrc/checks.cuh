// Checks of arguments that the C entries of sgemm_experts.h and sgemm_layers.h share.
#pragma once

#include "../../include/sgemm_experts.h"

#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

namespace sgemm_gb300 {

// Largest row, column or token count: tile arithmetic stays below 2^31.
constexpr int64_t kMaxSize = (int64_t(1) << 31) - 1024;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool bad_size(int64_t n) { return n < 0; }
inline bool too_large(int64_t n) { return n > kMaxSize; }
inline int64_t type_size(int type) { return type == SGEMM_F32 ? 4 : type == SGEMM_BF16 ? 2 : 0; }
inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Bytes from the first to past the last element of `batch` matrices, -1 if
// they would not fit 63 bits.
inline int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t size, int64_t batch = 1, int64_t stride = 0)
{
    if (rows <= 0 || cols <= 0 || batch <= 0) return 0;
    const __int128 e = ((__int128)(batch - 1) * stride + (__int128)(rows - 1) * ld + cols) * size;
    return e > (__int128)INT64_MAX ? -1 : (int64_t)e;
}

// The same of an 8-bit output: the quantisers store `piece` bytes of a row at a
// time, the last row's padding with its last values (rows start on 16 bytes).
inline int64_t span_fp8(int64_t rows, int64_t cols, int64_t ld, int64_t piece, int64_t batch = 1, int64_t stride = 0)
{
    return span(rows, ceil_div(cols, piece) * piece, ld, 1, batch, stride);
}

// The product's operands in 8 bits: 16-byte rows on a 16-byte base.
inline bool bad_fp8(const void *p, int64_t ld, int64_t cols) { return !p || !aligned(p, 16) || ld < cols || ld % 16 != 0; }

// An array of a call: where it lies, its extent, and the size of its elements.
struct Region {
    const void *p;
    int64_t bytes, size;
    template <class T>
    Region(const T *p, int64_t bytes) : Region(p, bytes, sizeof(T)) {}
    Region(const void *p, int64_t bytes, int64_t size) : p(p), bytes(bytes), size(size) {}
};

inline bool overlap(const Region &a, const Region &b)
{
    if (a.bytes <= 0 || b.bytes <= 0 || !a.p || !b.p) return false;
    const __int128 a0 = (__int128)reinterpret_cast<uintptr_t>(a.p), b0 = (__int128)reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// SGEMM_OK, or why a call must not run: a region that overflows, elements that
// do not lie on multiples of their size, an output that overlaps an input or
// another output.
template <int NOUT, int NIN>
int check_regions(const Region (&out)[NOUT], const Region (&in)[NIN])
{
    for (const Region &o : out)
        if (o.bytes < 0) return SGEMM_ERR_OVERFLOW;
    for (const Region &i : in)
        if (i.bytes < 0) return SGEMM_ERR_OVERFLOW;
    auto between = [](const Region &r) { return r.bytes > 0 && !aligned(r.p, (uintptr_t)r.size); };
    for (const Region &o : out)
        if (between(o)) return SGEMM_ERR_INVALID_VALUE;
    for (const Region &i : in)
        if (between(i)) return SGEMM_ERR_INVALID_VALUE;
    for (int a = 0; a < NOUT; ++a) {
        for (int b = 0; b < a; ++b)
            if (overlap(out[a], out[b])) return SGEMM_ERR_INVALID_VALUE;
        for (const Region &i : in)
            if (overlap(out[a], i)) return SGEMM_ERR_INVALID_VALUE;
    }
    return SGEMM_OK;
}

inline int launched(cudaError_t e)
{
    if (e == cudaSuccess) return SGEMM_OK;
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
}

}  // namespace sgemm_gb300
