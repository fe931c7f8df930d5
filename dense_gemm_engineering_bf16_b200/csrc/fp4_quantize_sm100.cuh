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
    bool saturated;     // NV: quotients past 6.375
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
        s.saturated = s.byte == 0x7Eu;
        if (!finite) s.byte = 0x7Fu;
    } else {
        // 6 = 1.5 * 2^2, so e = E - 127 - 2 for a magnitude 1.f * 2^(E - 127), one more where 1.f > 1.5
        const int b = static_cast<int>(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x400000u ? 1 : 0);
        s.byte = static_cast<uint32_t>(max(b, 0));
        s.by = 0.0f;
        s.saturated = false;
        s.inv = __uint_as_float((254u - s.byte) << 23);
        if (!finite) {
            s.byte = 0xFFu;
            s.inv = 0.0f;
        }
    }
    return s;
}

// Two fp32 numbers in one register pair, and their packed arithmetic.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Eight codes, the first in the lowest bits; past 6 they are 6.
__device__ __forceinline__ uint32_t e2m1_codes8(const float (&q)[8]) {
    uint32_t w;
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

// Eight values divided by their block's scale, as codes.  MX: exact (a power of
// two).  NV: the rounded product with the reciprocal may miss a quotient that
// lies halfway between two codes, where the last bit decides; one step of
// iterative refinement (the residual is exact in an fma) gives the rounded
// quotient (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  Where the scale has saturated, quotients are
// bounded first, so that the residual stays finite: all past 6 are a 6.  The
// method's exception, a divisor b = 2^k (1 - 2^-24), moves no code: x / b is then
// x 2^-k (1 + 2^-24 + ..), half a step beside a border only for x = 2^(k-2), whose
// refined quotient is 1/4 (1 + 2^-23), as it has to be; dividing such blocks cost 4 %.
template <bool NV>
__device__ __forceinline__ uint32_t fp4_codes8(const float *v, const Fp4Scale &s) {
    float q[8];
    if (NV && s.saturated) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            q[i] = fminf(fmaxf(v[i] * s.inv, -8.0f), 8.0f);
            q[i] = fmaf(fmaf(-q[i], s.by, v[i]), s.inv, q[i]);
        }
        return e2m1_codes8(q);
    }
    const uint64_t inv = f32x2(s.inv, s.inv), by = f32x2(-s.by, -s.by);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t x = f32x2(v[i], v[i + 1]);
        uint64_t r = mul_f32x2(x, inv);
        if (NV) r = fma_f32x2(fma_f32x2(r, by, x), inv, r);
        asm("mov.b64 {%0, %1}, %2;" : "=f"(q[i]), "=f"(q[i + 1]) : "l"(r));
    }
    return e2m1_codes8(q);
}

// Sixteen consecutive elements, as they are in memory.
template <int T>
struct Raw16 {
    uint32_t w[T == kF32 ? 16 : 8];
};

// WIDE: 32-byte aligned.
template <int T, bool WIDE>
__device__ __forceinline__ void load_raw16(const uint8_t *p, Raw16<T> &r) {
#pragma unroll
    for (int i = 0; i < (T == kF32 ? 16 : 8); i += 8) {
        if constexpr (WIDE) {
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(r.w[i]), "=r"(r.w[i + 1]), "=r"(r.w[i + 2]), "=r"(r.w[i + 3]), "=r"(r.w[i + 4]),
                           "=r"(r.w[i + 5]), "=r"(r.w[i + 6]), "=r"(r.w[i + 7])
                         : "l"(p + 4 * i));
        } else {
            const uint4 a = *reinterpret_cast<const uint4 *>(p + 4 * i), b = *reinterpret_cast<const uint4 *>(p + 4 * i + 16);
            r.w[i] = a.x, r.w[i + 1] = a.y, r.w[i + 2] = a.z, r.w[i + 3] = a.w;
            r.w[i + 4] = b.x, r.w[i + 5] = b.y, r.w[i + 6] = b.z, r.w[i + 7] = b.w;
        }
    }
}

// The largest magnitude (fp32 bits) and the values.  bf16: two at a time.
template <int T>
__device__ __forceinline__ uint32_t widen16(const Raw16<T> &r, float (&v)[16]) {
    if constexpr (T == kF32) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r.w[i]);
        return max_magnitude<16>(v);
    } else {
        uint32_t m = r.w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < 8; ++i) asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(r.w[i] & 0x7FFF7FFFu));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = __uint_as_float(r.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
        }
        return max(m << 16, m & 0xFFFF0000u);
    }
}

struct Fp4QuantizeArgs {
    const void *x;
    const float *g;         // null: 1
    uint8_t *q, *sf;
    int64_t M, K, ldx, ldq, tiles;   // tiles: scale tiles along K
};

// X stored K-major (M rows of K): VPT sixteens per thread, one NV block each or
// half an MX block; 4 neighbouring threads (MX: 8) hold the blocks of a word of
// scales.  A row takes blockDim.x threads in each of `parts` blocks; short rows
// share a block (blockDim.y).  8192 x 8192 from bf16: 30 us, 88 % of the copy rate
// (either format; 57 with eights of a warp's lanes, shuffles for the maxima and
// scalar arithmetic: the instructions, not memory, were the time), from fp32 45 us,
// 104 %; one row of 8192: 1.6 us.  32-byte loads where the rows' alignment allows.
template <int XT, bool NV, int VPT, bool WIDE>
__global__ void __launch_bounds__(256) fp4_quantize_kernel(Fp4QuantizeArgs a, unsigned parts) {
    wait_for_stream();
    const unsigned part = blockIdx.x % parts;
    const int64_t row = static_cast<int64_t>(blockIdx.x / parts) * blockDim.y + threadIdx.y;
    if (row >= a.M) return;   // whole warps
    const uint8_t *p = static_cast<const uint8_t *>(a.x) + row * a.ldx * elem_bytes<XT>;
    const int64_t first = 16 * (static_cast<int64_t>(part) * VPT * blockDim.x + threadIdx.x);
    Raw16<XT> r[VPT] = {};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t e = first + 16 * i * static_cast<int64_t>(blockDim.x);
        if (e < a.K) load_raw16<XT, WIDE>(p + e * elem_bytes<XT>, r[i]);
    }
    const float g = NV && a.g ? __ldcg(a.g) : 1.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t e = first + 16 * i * static_cast<int64_t>(blockDim.x);
        float v[16];
        uint32_t top = widen16<XT>(r[i], v);
        if (!NV) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        const Fp4Scale s = fp4_scale<NV>(top, g);
        constexpr int LANES = NV ? 1 : 2;       // of a block
        uint32_t word = e < a.K ? s.byte << (8 * (threadIdx.x / LANES & 3)) : 0u;
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, LANES);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * LANES);
        if (e < a.K) {
            *reinterpret_cast<uint2 *>(a.q + row * a.ldq + e / 2) =
                make_uint2(fp4_codes8<NV>(&v[0], s), fp4_codes8<NV>(&v[8], s));
            if (threadIdx.x % (4 * LANES) == 0)
                *reinterpret_cast<uint32_t *>(scale_word(a.sf, row, a.tiles, e / (64 * LANES))) = word;
        }
    }
}

// X stored MN-major (K rows of M: element (i, k) at X[k * ldx + i]).  A warp
// takes 32 K of 64 rows i, two per lane: 32 coalesced loads, then each lane
// holds whole blocks, without a shuffle.  The four warps of a block take 128
// consecutive K; their codes and scales meet in shared memory, from where
// each row i goes out as 64 bytes of codes and one (MX) or two words of scales.
// 8192 x 8192 from bf16: MX 28.1 us, 93 % of the copy rate, NV 36.9 with six blocks
// per SM (40.5 with five, 41.1 with eight); 4096 x 4096 NV 11.7; from fp32 45 to 46.5.
template <int XT, bool NV>
__global__ void __launch_bounds__(128, XT == kF32 ? 5 : NV ? 6 : 7) fp4_quantize_mn_kernel(Fp4QuantizeArgs a, unsigned i_tiles) {
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
        const float g = NV && a.g ? __ldcg(a.g) : 1.0f;
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
