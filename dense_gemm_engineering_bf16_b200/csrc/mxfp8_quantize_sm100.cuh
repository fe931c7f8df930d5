// MXFP8 encoding of a matrix: E4M3 codes and one E8M0 scale per 32
// consecutive K elements of each row, as gemm_mxfp8 reads them.  Bound by
// memory: each value is read once and its block stays in registers.
#pragma once
#include "rows.cuh"

namespace b200 {

// X stored K-major (M rows of K): VPT eights per thread.  A row (or a part of
// it: blockIdx.y) takes blockDim.x threads; short rows share a block
// (blockDim.y).
template <int XT, int VPT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const void *x, uint8_t *q, uint8_t *sf, int64_t M, int64_t K,
                                                          int64_t ldx, int64_t ldq) {
    constexpr bool SPLIT = XT == kF32;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= M) return;   // whole warps
    const uint8_t *p = static_cast<const uint8_t *>(x) + row * ldx * elem_bytes<XT>;
    Raw8<XT> r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        r[i] = load_raw8<XT, SPLIT>(p, first8<SPLIT>(threadIdx.x, blockIdx.y * VPT + i, blockDim.x), K);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float v[8];
        widen8<XT>(r[i], v);
        mx_store8<SPLIT>(v, first8<SPLIT>(threadIdx.x, blockIdx.y * VPT + i, blockDim.x), K, q + row * ldq,
                         sf + row * (K / 32));
    }
}

// X stored MN-major (K rows of M: element (i, k) at X[k * ldx + i]).  A warp
// takes 32 K of 64 rows i, two per lane: 32 coalesced loads, then each lane
// holds two whole blocks and writes each as 32 consecutive bytes.  The four
// warps of a block take 128 consecutive K, so that they fill whole 128-byte
// lines of codes together.
template <int XT>
__global__ void __launch_bounds__(128) mx_quantize_mn_kernel(const void *x, uint8_t *q, uint8_t *sf, int64_t M,
                                                             int64_t K, int64_t ldx, int64_t ldq, int64_t k_tiles) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) / k_tiles) * 64 + 2 * lane;
    const int64_t k0 = (static_cast<int64_t>(blockIdx.x) % k_tiles) * 128 + 32 * warp;
    if (k0 >= K || i >= M) return;
    const bool two = i + 1 < M;
    const uint8_t *p = static_cast<const uint8_t *>(x) + (k0 * ldx + i) * elem_bytes<XT>;
    const int64_t pitch = ldx * elem_bytes<XT>;
    float v[2][32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        const uint8_t *pk = p + k * pitch;
        if constexpr (XT == kF32) {
            if (two) {
                const float2 f = *reinterpret_cast<const float2 *>(pk);
                v[0][k] = f.x;
                v[1][k] = f.y;
            } else {
                v[0][k] = *reinterpret_cast<const float *>(pk);
                v[1][k] = 0.0f;
            }
        } else {
            const uint32_t w = two ? *reinterpret_cast<const uint32_t *>(pk) : *reinterpret_cast<const uint16_t *>(pk);
            v[0][k] = __uint_as_float(w << 16);
            v[1][k] = __uint_as_float(w & 0xFFFF0000u);
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (c == 1 && !two) break;
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) m = finite_max_bits(m, v[c][k]);
        const uint32_t byte = mx_scale_byte(m);
        const float inv = mx_inv_scale(byte);
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = e4m3_pair(v[c][4 * k], v[c][4 * k + 1], inv) | (e4m3_pair(v[c][4 * k + 2], v[c][4 * k + 3], inv) << 16);
        uint4 *d = reinterpret_cast<uint4 *>(q + (i + c) * ldq + k0);
        d[0] = make_uint4(w[0], w[1], w[2], w[3]);
        d[1] = make_uint4(w[4], w[5], w[6], w[7]);
        sf[(i + c) * (K / 32) + k0 / 32] = static_cast<uint8_t>(byte);
    }
}

}  // namespace b200
