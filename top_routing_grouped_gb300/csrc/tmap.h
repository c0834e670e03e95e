// tmap.h -- TMA tensor maps of row-major tensors (the weight-gradient outputs, the 8-bit products).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// 2-D fp32 row-major [rows, cols] tensor, boxes of [box_rows, 32] (128-byte rows) with
// 128-byte swizzle: the layout the TMA stores of the weight-gradient epilogue read from
// shared memory.  base 16-byte aligned, cols a multiple of 4.
cudaError_t make_tmap_f32_rows128(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows);

// 2-D row-major [rows, cols] tensor of 1-, 2- (bf16) or 4-byte (fp32) elements, boxes of
// [box_rows, 128 bytes] with 128-byte swizzle; a box past the tensor's edge reads zeros and
// stores nothing.  base 16-byte aligned, a row a multiple of 16 bytes.
cudaError_t make_tmap_rows128(CUtensorMap* m, const void* base, int esz, uint64_t rows, uint64_t cols, uint32_t box_rows);

}  // namespace moe
