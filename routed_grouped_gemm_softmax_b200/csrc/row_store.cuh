// row_store.cuh -- a warp's accumulator rows to global memory by whole row pieces.
//
// After tcgen05.ld a lane holds 32 columns of its own row.  Stored from there, one
// instruction touches 32 rows, 16 bytes each: 32 passes of the store unit, which a down
// item's few K stages do not hide (2048 tokens, k 6 of 64 experts, H 2048, fp32 rows: 27 of
// 163 us).  Turned in shared memory, it writes 4 rows of 128 bytes (fp32) or 8 of 64 (bf16).
// A warp without its 32 rows stores them from where they are: the turn costs the same for any
// number (16 rows a tile: 2 to 7% of the layer's time; 1024 rows an expert: 3 to 5% less).
#pragma once
#include <cstdint>

namespace moe {

constexpr int kRowStoreBytes = 4096;  // a warp's buffer, 16-byte aligned; null: rows are not turned

// Columns col .. col + 31 of the warp's rows, fp32: lane l has row l, which goes to row `to` of y (N
// columns) if l < rows.
__device__ __forceinline__ void store_rows_f32(uint8_t *buf, const uint32_t (&r)[32], float *y, int N, int col, int to,
                                               int rows, int lane)
{
    if (!buf || rows < 32) {
        if (lane < rows) {
            uint4 *dst = reinterpret_cast<uint4 *>(y + (size_t)to * N + col);
#pragma unroll
            for (int p = 0; p < 8; ++p) dst[p] = make_uint4(r[4 * p], r[4 * p + 1], r[4 * p + 2], r[4 * p + 3]);
        }
        return;
    }
#pragma unroll
    for (int p = 0; p < 8; ++p)  // piece p of row l at p ^ (l % 8): no bank twice on either side
        *reinterpret_cast<uint4 *>(buf + lane * 128 + ((p ^ (lane & 7)) * 16)) =
            make_uint4(r[4 * p], r[4 * p + 1], r[4 * p + 2], r[4 * p + 3]);
    __syncwarp();
#pragma unroll
    for (int it = 0; it < 8; ++it) {
        const int row = it * 4 + lane / 8, p = lane & 7;
        const uint4 v = *reinterpret_cast<const uint4 *>(buf + row * 128 + ((p ^ (row & 7)) * 16));
        const int at = __shfl_sync(0xffffffffu, to, row);
        if (row < rows) *reinterpret_cast<uint4 *>(y + (size_t)at * N + col + p * 4) = v;
    }
    __syncwarp();
}

// The same of bf16 pairs.
__device__ __forceinline__ void store_rows_bf16(uint8_t *buf, const uint32_t (&pk)[16], __nv_bfloat16 *y, int N, int col,
                                                int to, int rows, int lane)
{
    if (!buf || rows < 32) {
        if (lane < rows) {
            uint4 *dst = reinterpret_cast<uint4 *>(y + (size_t)to * N + col);
#pragma unroll
            for (int p = 0; p < 4; ++p) dst[p] = make_uint4(pk[4 * p], pk[4 * p + 1], pk[4 * p + 2], pk[4 * p + 3]);
        }
        return;
    }
#pragma unroll
    for (int p = 0; p < 4; ++p)
        *reinterpret_cast<uint4 *>(buf + lane * 64 + ((p ^ (lane >> 1 & 3)) * 16)) =
            make_uint4(pk[4 * p], pk[4 * p + 1], pk[4 * p + 2], pk[4 * p + 3]);
    __syncwarp();
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int row = it * 8 + lane / 4, p = lane & 3;
        const uint4 v = *reinterpret_cast<const uint4 *>(buf + row * 64 + ((p ^ (row >> 1 & 3)) * 16));
        const int at = __shfl_sync(0xffffffffu, to, row);
        if (row < rows) *reinterpret_cast<uint4 *>(y + (size_t)at * N + col + p * 8) = v;
    }
    __syncwarp();
}

}  // namespace moe
