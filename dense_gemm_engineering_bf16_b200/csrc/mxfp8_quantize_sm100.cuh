// MXFP8 encoding of a matrix: E4M3 codes and one E8M0 scale per 32
// consecutive K elements of each row, as gemm_mxfp8 reads them.  Bound by
// memory: each value is read once and its block stays in registers.
#pragma once
#include "rows.cuh"

namespace b200 {

// X stored K-major (M rows of K): VPT eights per thread.  A row takes
// blockDim.x threads in each of `parts` blocks; short rows share a block
// (blockDim.y).  8192 x 8192: 34.2 us from bf16 (91 % of the copy rate), 50.9 from
// fp32 (101 %); 1000 x 8192 bf16: 5.0 us, which is L2's rate and the launch.
template <int XT, int VPT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const void *x, uint8_t *q, uint8_t *sf, int64_t M, int64_t K,
                                                          int64_t ldx, int64_t ldq, unsigned parts) {
    constexpr bool SPLIT = XT == kF32;
    wait_for_stream();
    const unsigned part = blockIdx.x % parts;
    const int64_t row = static_cast<int64_t>(blockIdx.x / parts) * blockDim.y + threadIdx.y;
    if (row >= M) return;   // whole warps
    const uint8_t *p = static_cast<const uint8_t *>(x) + row * ldx * elem_bytes<XT>;
    Raw8<XT> r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        r[i] = load_raw8<XT, SPLIT>(p, first8<SPLIT>(threadIdx.x, part * VPT + i, blockDim.x), K);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float v[8];
        widen8<XT>(r[i], v);
        mx_store8<SPLIT>(v, first8<SPLIT>(threadIdx.x, part * VPT + i, blockDim.x), K, q + row * ldq,
                         sf + row * (K / 32));
    }
}

// X stored MN-major (K rows of M: element (i, k) at X[k * ldx + i]).  A warp
// takes 32 K of 64 rows i, two per lane: 32 coalesced loads, then each lane
// holds two whole blocks, without a shuffle.  The four warps of a block take
// 128 consecutive K; their codes and scales meet in shared memory, from where
// each row i goes out as one 128-byte line of codes and its four scales
// together.  Neighbouring blocks read neighbouring pieces of the same rows of X.
// 8192 x 8192 bf16: 33.1 us, 94 % of the copy rate (35.0 with neighbours along K;
// written straight from the lanes, 32 bytes of a row each and single scale
// bytes, 58); the registers are held to seven blocks per SM (72, with 12 bytes
// spilled; eight blocks spill more: 43.1).  From fp32, five blocks: 50.8 us, 101 %.
template <int XT>
__global__ void __launch_bounds__(128, XT == kF32 ? 5 : 7) mx_quantize_mn_kernel(const void *x, uint8_t *q, uint8_t *sf, int64_t M,
                                                             int64_t K, int64_t ldx, int64_t ldq, unsigned i_tiles) {
    constexpr int kPitch = 128 + 16;
    __shared__ __align__(16) uint8_t tile[64 * kPitch];
    __shared__ __align__(4) uint8_t scales[64][4];
    wait_for_stream();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x % i_tiles) * 64;
    const int64_t kb = static_cast<int64_t>(blockIdx.x / i_tiles) * 128, k0 = kb + 32 * warp;
    const int64_t left = M - i0 - 2 * lane;      // rows from this lane's first on
    if (k0 < K && left > 0) {
        const uint8_t *p = static_cast<const uint8_t *>(x) + (k0 * ldx + i0 + 2 * lane) * elem_bytes<XT>;
        const int64_t pitch = ldx * elem_bytes<XT>;
        float v[2][32];
        if (left > 1) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                if constexpr (XT == kF32) {
                    const float2 f = *reinterpret_cast<const float2 *>(p + k * pitch);
                    v[0][k] = f.x;
                    v[1][k] = f.y;
                } else {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(p + k * pitch);
                    v[0][k] = __uint_as_float(w << 16);
                    v[1][k] = __uint_as_float(w & 0xFFFF0000u);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                if constexpr (XT == kF32)
                    v[0][k] = *reinterpret_cast<const float *>(p + k * pitch);
                else
                    v[0][k] = __uint_as_float(
                        static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(p + k * pitch)) << 16);
                v[1][k] = 0.0f;
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t byte = mx_scale_byte(finite_max<32>(v[c]));
            const float inv = mx_inv_scale(byte);
            uint4 *d = reinterpret_cast<uint4 *>(&tile[(2 * lane + c) * kPitch + 32 * warp]);
            d[0] = make_uint4(e4m3_codes4(&v[c][0], inv), e4m3_codes4(&v[c][4], inv), e4m3_codes4(&v[c][8], inv),
                              e4m3_codes4(&v[c][12], inv));
            d[1] = make_uint4(e4m3_codes4(&v[c][16], inv), e4m3_codes4(&v[c][20], inv), e4m3_codes4(&v[c][24], inv),
                              e4m3_codes4(&v[c][28], inv));
            scales[2 * lane + c][warp] = static_cast<uint8_t>(byte);
        }
    }
    __syncthreads();
    const int rows = static_cast<int>(min(M - i0, static_cast<int64_t>(64)));
    const int64_t k_left = K - kb;               // a multiple of 32
    const int col = 16 * (threadIdx.x % 8);
#pragma unroll
    for (int r = threadIdx.x / 8; r < 64; r += 16)
        if (r < rows && col < k_left)
            *reinterpret_cast<uint4 *>(q + (i0 + r) * ldq + kb + col) =
                *reinterpret_cast<const uint4 *>(&tile[r * kPitch + col]);
    const int r = threadIdx.x;
    if (r < rows) {
        uint8_t *d = sf + (i0 + r) * (K / 32) + kb / 32;
        if (k_left >= 128 && (reinterpret_cast<uintptr_t>(d) & 3) == 0) {
            *reinterpret_cast<uint32_t *>(d) = *reinterpret_cast<const uint32_t *>(scales[r]);
        } else {
            for (int j = 0; j < 4 && 32 * j < k_left; ++j) d[j] = scales[r][j];
        }
    }
}

}  // namespace b200
