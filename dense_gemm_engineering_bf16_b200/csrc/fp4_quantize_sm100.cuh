// 4-bit floating-point encoding of a matrix: E2M1 codes, two a byte, and one
// scale per block of consecutive K elements of each row, in the tiles that
// gemm_fp4's tensor cores take them in.  Bound by memory: each value is read
// once and its block stays in registers.
//
//   MX  blocks of 32, scale 2^e, the smallest with |v| <= 6 * 2^e (6 is the
//       largest E2M1 value), as the MXFP8 encoding in rows.cuh
//   NV  blocks of 16 under a scale g of the whole tensor: s = E4M3(max |v| / (6 g)),
//       at least 2^-9 (the smallest), at most 448; a code is v / (s g)
//
// rounded to nearest even, past 6 to 6.  E2M1 has no NaN: a block with a NaN or
// an infinity gets the scale's NaN, which makes its products NaN.
#pragma once
#include "rows.cuh"

namespace b200 {

// Bytes of a scale tile (128 rows x 4 blocks): row r of the tile has its four
// bytes at 16 (r % 32) + 4 (r / 32), the layout that tcgen05.cp puts into tensor
// memory; tiles of 128 rows follow one another along K.
constexpr int kScaleTile = 512;

template <bool NV>
constexpr int kFp4Block = NV ? 16 : 32;

__device__ __forceinline__ uint8_t *scale_word(uint8_t *sf, int64_t row, int64_t tiles, int64_t tile) {
    return sf + ((row >> 7) * tiles + tile) * kScaleTile + (row & 31) * 16 + (row >> 5 & 3) * 4;
}

// Magnitude bits, in whose order NaN comes after infinity and that after the
// finite values.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int N>
__device__ __forceinline__ uint32_t max_magnitude(const float *v) {
    uint32_t m = magnitude(v[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) m = max(m, magnitude(v[i]));
    return m;
}

// A block's scale byte from its largest magnitude, and what its values are
// divided by: `by` (MX: a power of two) with its reciprocal.
struct Fp4Scale {
    uint32_t byte;
    float by, inv;
};

template <bool NV>
__device__ __forceinline__ Fp4Scale fp4_scale(uint32_t top, float g) {
    const bool finite = top < 0x7F800000u;
    Fp4Scale s;
    if constexpr (NV) {
        uint16_t b;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.0f), "f"(__fdiv_rn(__uint_as_float(top), 6.0f * g)));
        s.byte = max(static_cast<uint32_t>(b), 1u);
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(s.byte)));
        float f;
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
        s.by = f * g;
        s.inv = __frcp_rn(s.by);
        if (!finite) s.byte = 0x7Fu;
    } else {
        // 6 = 1.5 * 2^2, so e = E - 127 - 2 for a magnitude 1.f * 2^(E - 127), one more where 1.f > 1.5
        const int b = static_cast<int>(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x400000u ? 1 : 0);
        s.byte = static_cast<uint32_t>(max(b, 0));
        s.by = 0.0f;
        s.inv = __uint_as_float((254u - s.byte) << 23);
        if (!finite) {
            s.byte = 0xFFu;
            s.inv = 0.0f;
        }
    }
    return s;
}

// v divided by the scale.  MX: exact (a power of two).  NV: the rounded product
// with the reciprocal may miss a quotient that lies halfway between two codes,
// where the last bit decides; one step of iterative refinement (the residual is
// exact in an fma) gives the rounded quotient (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  Bounded
// first, so that the residual stays finite: every quotient past 6 is a 6.
template <bool NV>
__device__ __forceinline__ float fp4_quotient(float v, const Fp4Scale &s) {
    float q = v * s.inv;
    if constexpr (NV) {
        q = fminf(fmaxf(q, -8.0f), 8.0f);
        q = fmaf(fmaf(-q, s.by, v), s.inv, q);
    }
    return q;
}

// Eight codes, the first in the lowest bits; past 6 they are 6.
template <bool NV>
__device__ __forceinline__ uint32_t fp4_codes8(const float *v, const Fp4Scale &s) {
    uint32_t w;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fp4_quotient<NV>(v[i], s);
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return w;
}

template <bool NV>
__device__ __forceinline__ uint16_t fp4_codes4(const float *v, const Fp4Scale &s) {
    uint16_t w;
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = fp4_quotient<NV>(v[i], s);
    asm("{\n\t.reg .b8 a, b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "mov.b16 %0, {a, b};\n\t}"
        : "=h"(w)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]));
    return w;
}

// Encodes a group of values that the warp's lanes hold side by side, E (8 or 4)
// each from element e on, those past K as zeros: a block is B / E neighbouring
// lanes, four blocks' scales a word.  All 32 lanes call it.
template <bool NV, int E>
__device__ __forceinline__ void fp4_store(const float *v, int64_t e, int64_t K, float g, uint8_t *q, uint8_t *sf,
                                          int64_t row, int64_t tiles) {
    constexpr int LANES = kFp4Block<NV> / E;
    uint32_t top = max_magnitude<E>(v);
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    const Fp4Scale s = fp4_scale<NV>(top, g);
    const int lane = threadIdx.x & 31;
    uint32_t word = e < K ? s.byte << (8 * (lane / LANES & 3)) : 0u;
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, LANES);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * LANES);
    if (e < K) {
        if constexpr (E == 8) *reinterpret_cast<uint32_t *>(q + e / 2) = fp4_codes8<NV>(v, s);
        else *reinterpret_cast<uint16_t *>(q + e / 2) = fp4_codes4<NV>(v, s);
        if (lane % (4 * LANES) == 0)
            *reinterpret_cast<uint32_t *>(scale_word(sf, row, tiles, e / (4 * kFp4Block<NV>))) = word;
    }
}

struct Fp4QuantizeArgs {
    const void *x;
    const float *g;         // null: 1
    uint8_t *q, *sf;
    int64_t M, K, ldx, ldq, tiles;   // tiles: scale tiles along K
};

// X stored K-major (M rows of K): VPT eights per thread.  A row takes
// blockDim.x threads in each of `parts` blocks; short rows share a block
// (blockDim.y).
template <int XT, bool NV, int VPT>
__global__ void __launch_bounds__(256) fp4_quantize_kernel(Fp4QuantizeArgs a, unsigned parts) {
    constexpr bool SPLIT = XT == kF32;
    wait_for_stream();
    const unsigned part = blockIdx.x % parts;
    const int64_t row = static_cast<int64_t>(blockIdx.x / parts) * blockDim.y + threadIdx.y;
    if (row >= a.M) return;   // whole warps
    const uint8_t *p = static_cast<const uint8_t *>(a.x) + row * a.ldx * elem_bytes<XT>;
    uint8_t *q = a.q + row * a.ldq;
    Raw8<XT> r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        r[i] = load_raw8<XT, SPLIT>(p, first8<SPLIT>(threadIdx.x, part * VPT + i, blockDim.x), a.K);
    const float g = NV && a.g ? __ldg(a.g) : 1.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float v[8];
        widen8<XT>(r[i], v);
        const int64_t e = first8<SPLIT>(threadIdx.x, part * VPT + i, blockDim.x);
        if constexpr (SPLIT) {
            fp4_store<NV, 4>(&v[0], e, a.K, g, q, a.sf, row, a.tiles);
            fp4_store<NV, 4>(&v[4], e + at8<true>(4), a.K, g, q, a.sf, row, a.tiles);
        } else {
            fp4_store<NV, 8>(v, e, a.K, g, q, a.sf, row, a.tiles);
        }
    }
}

// X stored MN-major (K rows of M: element (i, k) at X[k * ldx + i]).  A warp
// takes 32 K of 64 rows i, two per lane: 32 coalesced loads, then each lane
// holds whole blocks, without a shuffle.  The four warps of a block take 128
// consecutive K; their codes and scales meet in shared memory, from where
// each row i goes out as 64 bytes of codes and one (MX) or two words of scales.
template <int XT, bool NV>
__global__ void __launch_bounds__(128) fp4_quantize_mn_kernel(Fp4QuantizeArgs a, unsigned i_tiles) {
    constexpr int kPitch = 64 + 16, B = kFp4Block<NV>, WORDS = NV ? 2 : 1;
    __shared__ __align__(16) uint8_t tile[64 * kPitch];
    __shared__ __align__(8) uint8_t scales[64][4 * WORDS];
    wait_for_stream();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x % i_tiles) * 64;
    const int64_t kb = static_cast<int64_t>(blockIdx.x / i_tiles) * 128, k0 = kb + 32 * warp;
    const int64_t left = a.M - i0 - 2 * lane;      // rows from this lane's first on
    if (left > 0) {
        float v[2][32];
        if (k0 < a.K) {
            const uint8_t *p = static_cast<const uint8_t *>(a.x) + (k0 * a.ldx + i0 + 2 * lane) * elem_bytes<XT>;
            const int64_t pitch = a.ldx * elem_bytes<XT>;
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
        }
        const float g = NV && a.g ? __ldg(a.g) : 1.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (k0 < a.K) {
                uint32_t w[4];
#pragma unroll
                for (int b = 0; b < 32 / B; ++b) {
                    const Fp4Scale s = fp4_scale<NV>(max_magnitude<B>(&v[c][B * b]), g);
#pragma unroll
                    for (int i = 0; i < B / 8; ++i) w[B / 8 * b + i] = fp4_codes8<NV>(&v[c][B * b + 8 * i], s);
                    scales[2 * lane + c][32 / B * warp + b] = static_cast<uint8_t>(s.byte);
                }
                *reinterpret_cast<uint4 *>(&tile[(2 * lane + c) * kPitch + 16 * warp]) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int b = 0; b < 32 / B; ++b) scales[2 * lane + c][32 / B * warp + b] = 0;
            }
        }
    }
    __syncthreads();
    const int rows = static_cast<int>(min(a.M - i0, static_cast<int64_t>(64)));
    const int64_t k_left = a.K - kb;               // a multiple of 32
    const int col = 16 * (threadIdx.x % 4);
#pragma unroll
    for (int r = threadIdx.x / 4; r < 64; r += 32)
        if (r < rows && 2 * col < k_left)
            *reinterpret_cast<uint4 *>(a.q + (i0 + r) * a.ldq + kb / 2 + col) =
                *reinterpret_cast<const uint4 *>(&tile[r * kPitch + col]);
    const int r = threadIdx.x % 64, w = threadIdx.x / 64;
    if (w < WORDS && r < rows && 4 * B * w < k_left)
        *reinterpret_cast<uint32_t *>(scale_word(a.sf, i0 + r, a.tiles, kb / (4 * B) + w)) =
            *reinterpret_cast<const uint32_t *>(&scales[r][4 * w]);
}

}  // namespace b200
