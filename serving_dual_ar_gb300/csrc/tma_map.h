// Tensor-map (TMA descriptor) encoding shared by the tcgen05 kernels.
#pragma once

#include <cuda.h>

namespace s2 {

// 2-D bf16 map over [rows, cols] (cols contiguous, row pitch ld elements,
// ld * 2 a multiple of 16 bytes, base 16-byte aligned) with a box of
// box_rows x 64 columns and 128-byte swizzle; rows past the end read 0.
// False when the driver entry point is missing or the encoding is refused.
bool tma_map_bf16_2d(CUtensorMap* m, const void* base, long long rows, int cols, int ld, int box_rows);

// Pool of 8-bit KV pages [n_pages][2][Hkv][16][hd] as a 5-D byte map whose box
// is one head's 16 key rows and 16 value rows of a page, swizzled over the
// row's length (128 or 64 bytes).
bool tma_map_kv8(CUtensorMap* m, const void* kv, int n_pages, int Hkv, int hd);

// 4-bit weights [rows][cols / 2 bytes], cols a multiple of 128, 32-byte aligned:
// a box of 128 rows x 128 values arrives as 128-byte rows with 8 of each 16 bytes
// in use, 128-byte swizzle.
bool tma_map_w4(CUtensorMap* m, const void* codes, long long rows, int cols);
// Byte rows [rows][cols], pitch ld (a multiple of 16): boxes of box_rows x 128
// bytes, 128-byte swizzle; bytes past the end read 0.
bool tma_map_u8_2d(CUtensorMap* m, const void* base, long long rows, int cols, long long ld, int box_rows);

}  // namespace s2
