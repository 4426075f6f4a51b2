// Rows of a matrix as windows of whole 16-byte chunks, the form in which the norm's
// rings copy them: by address, so that any length and pitch will do.  Plain C++, for
// the host side, the kernels and a test without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MBT_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MBT_HOST_DEVICE inline
#endif

namespace mbt {

struct RowWindow {
    int lead;                // bytes from the window's first to the row's
    int64_t start;           // bytes from the matrix to the window
    int bytes;               // copied
};

// The first row whose last chunk is the matrix's own last one, and in part beyond
// it.  That chunk is not copied (the bytes after the matrix may be nobody's); the
// rows from here on take it by elements.  With a pitch of 16 bytes or more that is at
// most the last row; of shorter rows several can end in the chunk.  M rows of
// row_bytes bytes, ld bytes apart.
inline int64_t first_tail_row(int64_t M, int64_t row_bytes, int64_t ld) {
    const int64_t end = (M - 1) * ld + row_bytes, whole = end & ~int64_t{15};
    if (whole == end) return M;
    return whole < row_bytes ? 0 : (whole - row_bytes) / ld + 1;
}

// tail: first_tail_row of the matrix.  phased: rows may start inside a chunk.
MBT_HOST_DEVICE RowWindow row_window(int64_t row, int64_t tail, int row_bytes, int64_t ld, bool phased) {
    RowWindow w;
    const int64_t at = row * ld;
    w.lead = phased ? static_cast<int>(at & 15) : 0;
    w.start = at - w.lead;
    const int need = w.lead + row_bytes;
    w.bytes = row >= tail ? need & ~15 : (need + 15) & ~15;
    return w;
}

}  // namespace mbt
