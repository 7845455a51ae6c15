// row_phase.h -- rows that do not all start on 16-byte boundaries.  Internal
// to libgbnorm.so.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gbn {

// Rows whose starts are not all on 16 bytes.  Row r starts shift(r) elements
// after a 16-byte boundary, shift(r) = (shift0 + r * shift_step) mod V with
// V elements to 16 bytes; rows `phases` apart have the same shift.  CTA b
// takes rows b, b + G, ... with G a multiple of `phases`, so its threads'
// columns stay the same from row to row.
__host__ __device__ inline int row_shift(int64_t row, int shift0, int shift_step, int V) {
    return static_cast<int>((shift0 + row * shift_step) & (V - 1));
}

}  // namespace gbn
