// norm_rows.h -- which columns of a row a thread of the layer norm has, and which
// of its pieces may be loaded whole.  Plain C++, so that the index arithmetic also
// compiles for the host, where a test walks it.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FFTC_HD __host__ __device__ __forceinline__
#else
#define FFTC_HD inline
#endif

namespace fftc {
namespace ln {

// Elements from the start of row r to the end of the tensor, as far as they matter to a piece.
FFTC_HD int to_end(int64_t r, int64_t rows, int C) {
    const int64_t n = (rows - r) * C;
    return n < (1 << 30) ? (int)n : 1 << 30;
}

// The pieces of a thread: columns first(i) .. first(i) + V - 1 of its rows.
template <int V, int TPR, bool OFF>
struct Pieces {
    int lane, off, C;  // off: elements between the 16-byte boundary and the row
    FFTC_HD int first(int i) const { return (lane + i * TPR) * V - (OFF ? off : 0); }
    FFTC_HD bool any(int i) const { return first(i) < C; }
    FFTC_HD bool inside(int i) const { return !OFF || (first(i) >= 0 && first(i) + V <= C); }
    FFTC_HD bool has(int c) const { return (unsigned)c < (unsigned)C; }
    // Loaded as 16 bytes: a piece at a row's end as well, its other elements being a neighbouring row's (one or, with C
    // below V, several), but not where it goes on behind the tensor, `end` elements from the row's start.
    FFTC_HD bool whole(int i, int end) const { return !OFF || first(i) + V <= end; }
};
template <int V, bool OFF>
FFTC_HD int offset(int64_t row, int C) {
    return OFF ? (int)((uint64_t)row * (uint64_t)C % V) : 0;
}

}  // namespace ln
}  // namespace fftc
