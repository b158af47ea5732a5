// The rows that a thread of a row-wise kernel works on: a block holds rpb =
// threads / tpr rows at a time, tpr threads to each, and walks the rows gridDim
// steps apart.  All threads of a block go round equally often, past the last row
// too, since they shuffle and wait for one another on the way; a thread whose row
// is none (row >= rows) does it with zeros.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MGS_ROWS_FN __host__ __device__ __forceinline__
#else
#define MGS_ROWS_FN inline
#endif

namespace mgs {

struct RowWalk {
    int64_t base, row, step;  // the block's first row, this thread's, and from one round to the next
    MGS_ROWS_FN RowWalk(unsigned block, unsigned blocks, unsigned thread, unsigned threads, int tpr) {
        const int64_t rpb = int(threads) / tpr;
        base = block * rpb, row = base + int(thread) / tpr, step = blocks * rpb;
    }
    MGS_ROWS_FN bool more(int64_t rows) const { return base < rows; }
    MGS_ROWS_FN void next() { base += step, row += step; }
};

}  // namespace mgs
