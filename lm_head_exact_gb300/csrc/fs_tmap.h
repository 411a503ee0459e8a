// TMA tensor-map encoding for the tensor-core kernels (host side).
#pragma once

#include <cuda.h>

#include <cstdint>

namespace fs {

// Encode a 2-D tensor map over a bf16 matrix [rows, cols] whose rows lie
// `pitch` elements apart (a multiple of 8), in boxes of box_cols elements (the
// contiguous direction) by box_rows rows, stored in shared memory with the
// 128-byte swizzle that the tcgen05 descriptors expect: a K-major operand's
// boxes, or, 64 columns by k rows, those of an operand stored along its M or N
// axis.  Out-of-range parts of a box read as zero and are not stored.  Returns
// false if the driver entry point is unavailable or rejects the description.
bool encode_rows_bf16(CUtensorMap* tm, const void* base, int64_t rows, int64_t cols, int64_t pitch, int box_cols,
                      int box_rows);

// The same over a matrix without gaps, d elements a row.
bool encode_kmajor_bf16(CUtensorMap* tm, const void* base, int64_t rows, int64_t d, int box_cols, int box_rows);

}  // namespace fs
