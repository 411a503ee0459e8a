// Tensor-map encoding for the LM head's training products (host side).
#pragma once

#include <cuda.h>

#include <cstdint>

namespace fs {

// A 2-D tensor map over a bf16 matrix [rows, cols] whose rows lie `pitch`
// elements apart (a multiple of 8), in boxes of 64 columns by box_rows rows
// stored with the 128-byte swizzle: a K-major operand's boxes, or, 64 columns by
// k rows, those of an operand stored along its M or N axis.  Out-of-range
// parts of a box read as zero and are not stored.  False if the driver entry
// point is unavailable or rejects the description.
bool encode_rows_bf16(CUtensorMap* tm, const void* base, int64_t rows, int64_t cols, int64_t pitch, int box_rows);

}  // namespace fs
