// Output tiles of the large products: accumulator columns to bf16 rows in
// memory.  A thread holds 64 columns of one row; stored from there, a warp's
// every instruction would touch 16 bytes in each of 32 rows.  The warp passes
// 32 rows x 64 columns through shared memory instead (128B swizzle, so neither
// side meets bank conflicts) and a bulk tensor copy takes them out in whole
// 128-byte lines, clipped at the matrix's ends; two warps share a quarter of the
// lanes.  The FP4 product of 7168 x 5120 x 1024, mostly epilogue: 51 us with
// direct stores from four warps, 45 through the boxes, 31 with eight warps.
#pragma once
#include "kernels.h"
#include "ptx.cuh"

namespace fp4attn {

constexpr int STORE_WARPS = 8;  // two for each quarter of the lanes, a half of the columns each
constexpr uint32_t STORE_BOX = 32 * 128;  // bytes of 32 rows x 64 columns
constexpr uint32_t STORE_BYTES = STORE_WARPS * STORE_BOX;

// bf16 matrix [rows][cols] in boxes of 32 rows x 64 columns.
inline bool make_store_map(CUtensorMap* m, void* base, int64_t rows, int64_t cols, int64_t ld) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)ld * 2};
    const uint32_t box[2] = {64, 32};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// One warp's box, on a 1024-byte boundary: this lane's 64 values (as 32 bf16
// pairs) go to row `row` + lane, columns from `col`.
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t box, const uint32_t (&w)[32], int row, int col,
                                          int rows, int cols, int lane) {
    if (lane == 0) bulk_wait_read<0>();  // the copy before has left the box
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
        st_shared16(box + 128u * lane + 16u * (uint32_t)(j ^ (lane & 7)),
                    make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (row < rows && col < cols) tma_store_2d(map, col, row, box);
        bulk_commit();
    }
}
// Before the warp's shared memory goes.
__device__ __forceinline__ void store_box_finish(int lane) {
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
}

}  // namespace fp4attn
