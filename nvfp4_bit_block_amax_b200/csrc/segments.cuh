// segments.cuh -- expert segments of sorted rows, as the products read them.
//
// offsets and counts are device data that nothing has checked: wherever they
// are read they are clamped to 128-aligned ranges inside [0, limit), so that
// whatever they held, no access goes out of bounds.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace nvfp4 {

__device__ __forceinline__ int segment_start(const int* offsets, int e, int limit) {
    return min(max(offsets[e], 0), limit) & ~127;
}
__device__ __forceinline__ int segment_end(const int* offsets, const int* counts, int e, int limit) {   // of the rows in use
    const int start = segment_start(offsets, e, limit);
    return start + min(max(counts[e], 0), max(segment_start(offsets, e + 1, limit) - start, 0));
}

// Rows first .. last-1 of a matrix become zeros, one warp to a row; the rows
// are dealt to `workers` warps.  Rows start on 16-byte boundaries.
__device__ __forceinline__ void zero_rows(void* base, int64_t row_bytes, int64_t ld_bytes, int first, int last, int worker,
                                          int workers, int lane) {
    for (int64_t r = (int64_t)first + worker; r < last; r += workers) {
        uint8_t* q = static_cast<uint8_t*>(base) + r * ld_bytes;
        for (int64_t b = 16 * lane; b + 16 <= row_bytes; b += 512) *reinterpret_cast<uint4*>(q + b) = make_uint4(0, 0, 0, 0);
        const int64_t b = row_bytes / 16 * 16 + 2 * lane;
        if (b < row_bytes) *reinterpret_cast<uint16_t*>(q + b) = 0;
    }
}

}  // namespace nvfp4
