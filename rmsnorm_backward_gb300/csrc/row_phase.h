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

// Copies to a stage the elements of a tensor's first or last row [s, s + n) of
// whose first or last 16 bytes some lie outside the tensor; the bytes [x, y)
// are left for a bulk copy.  Out of line, as it is for two rows of a tensor;
// inlined the time is the same (27711x2202 bf16 to int8 69 us against 70, by 128
// columns 81 against 82).
template <typename T>
__device__ __noinline__ uint2 copy_end_row(T *dst, const T *src, const T *base, const T *end, int s, int n, uint32_t bytes) {
    uint32_t from = 0, to = bytes;
    if (src < base) from = 16;
    if (src + bytes / sizeof(T) > end) to = bytes - 16;
    for (int c = s; c < s + n && c < static_cast<int>(from / sizeof(T)); ++c) dst[c] = src[c];
    for (int c = max(static_cast<int>(to / sizeof(T)), s); c < s + n; ++c) dst[c] = src[c];
    return make_uint2(from, to);
}

}  // namespace gbn
