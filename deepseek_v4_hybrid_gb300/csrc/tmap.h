// Host helpers for TMA tensor maps (driver entry point fetched through the runtime, so the library
// needs no link-time dependency on libcuda) and the device's SM count.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dsv4 {

// 2-D bf16 tensor [rows, cols] (cols innermost, rows `cols * 2` bytes apart), box
// [box_rows, box_cols] with 128-byte swizzle (box_cols * 2 must be 128).
cudaError_t make_tmap_2d_bf16(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols,
                              uint32_t box_rows);

// 2-D tensor of `rows` rows of `cols` elements of type `dt`, consecutive rows `row_bytes` apart (a
// row may be wider than the mapped columns: a column range of packed records), box
// [box_rows, box_cols], swizzle `sw`.  Out-of-range rows read as zeros.
cudaError_t make_tmap_2d(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t cols, uint64_t rows,
                         uint64_t row_bytes, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle sw);

// 4-D bf16 tensor [d3, d2, d1, d0] (d0 innermost and contiguous; the others `s1`, `s2`, `s3` bytes apart), box of
// [1, b2, b1, b0] elements with 128-byte swizzle (b0 * 2 must be 128).  Elements out of range read as zeros.
cudaError_t make_tmap_4d_bf16(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t d3,
                              uint64_t s1, uint64_t s2, uint64_t s3, uint32_t b0, uint32_t b1, uint32_t b2);

// Multiprocessor count of the current device.
int num_sms();

// Sets the maximum dynamic shared memory of kernel `fn` to `bytes` on the current device, once per
// device (function attributes belong to each device's context); thread safe.
cudaError_t ensure_max_dynamic_smem(const void* fn, int bytes);

}  // namespace dsv4
