// TMA descriptors of packed codes (gemm.cu).
#pragma once

#include <cstdint>
#include <cuda.h>

namespace vlaq {

// 2-D byte tensor [rows, row_bytes] with the given pitch, box 128 x box_rows,
// 128-byte swizzle, zero fill out of bounds.  False when it cannot be encoded.
bool make_map(CUtensorMap* map, const void* base, uint64_t row_bytes, uint64_t rows, uint64_t pitch,
              uint32_t box_rows);

// bf16 tensor [rows, cols] in tiles of 64 columns x 32 rows (128-byte rows),
// 128-byte swizzle.  Needs a 16-byte aligned base and cols % 8 == 0.
bool make_out_map(CUtensorMap* map, void* base, uint64_t cols, uint64_t rows);
// The same to read, in tiles of 64 columns x box_rows rows.
bool make_bf16_map(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows);

}  // namespace vlaq
