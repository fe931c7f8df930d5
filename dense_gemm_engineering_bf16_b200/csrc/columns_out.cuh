// Write-back of products whose accumulator lies the other way round than C: a
// TMEM lane is a column of C, a TMEM column one of its rows.  A warp holds 32
// columns of C; each of its stores covers consecutive columns of a row.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "rows.cuh"

namespace b200 {

// W rows of C (from `c` on, the row of v[0], `ld` elements apart, the first
// `rows` of them written) x the warp's 32 columns, of which this lane holds
// column `col`: C = v + beta * C, rounded once.  Rows are 4-byte aligned (16 in
// fact) and the warp's first column is even.  bf16: neighbouring lanes trade
// halves, so that each holds two columns of one row and a store writes two rows
// of 64 bytes; half as many stores as with 16 bits a lane.
template <int W>
__device__ __forceinline__ void store_columns(void *c, int64_t ld, int rows, int col, int cols, bool f32, float beta,
                                              float (&v)[W]) {
    const bool mine = col < cols;
    if (f32) {
        float *p = static_cast<float *>(c) + col;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (j < rows && mine) {
                if (beta != 0.0f) v[j] = fmaf(beta, *p, v[j]);
                *p = v[j];
            }
            p += ld;
        }
        return;
    }
    if (beta != 0.0f) {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(c) + col;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (j < rows && mine) v[j] = fmaf(beta, __bfloat162float(*p), v[j]);
            p += ld;
        }
        __syncwarp();   // a neighbour may overwrite what this lane read
    }
    const bool odd = col & 1;
    uint16_t *p = static_cast<uint16_t *>(c) + (odd ? ld : 0) + (col & ~1);
    const bool pair = (col | 1) < cols, single = (col & ~1) < cols;
#pragma unroll
    for (int j = 0; j < W; j += 2) {
        const uint32_t own = pack_bf16x2(v[j], v[j + 1]);
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
        const uint32_t w = odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
        if (j + (odd ? 1 : 0) < rows) {
            if (pair) *reinterpret_cast<uint32_t *>(p) = w;
            else if (single) *p = static_cast<uint16_t>(w);
        }
        p += 2 * ld;
    }
}

}  // namespace b200
