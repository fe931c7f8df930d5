// Row-wise building blocks of the operators around the products: eight
// elements (bf16 or fp32) per thread and step, fixed-order sums, and the MXFP8
// encoding of 32 consecutive values.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

namespace b200 {

// Element types, numbered as gemm_out_t; kNone: no such operand.
constexpr int kF32 = 0, kBF16 = 1, kNone = 2;

template <int T>
constexpr int elem_bytes = T == kF32 ? 4 : 2;

// Eight elements of a row, as they are in memory: a thread's share of one step.
// With SPLIT they are two groups of four, 128 elements apart, so that each
// load or store instruction of a warp covers consecutive bytes when an
// operand is fp32 (eight consecutive fp32 per thread would touch every
// 32-byte sector twice); without it they are consecutive, one 16-byte access
// of bf16.  e is the first one's index; element j of the eight is at
// e + at8<SPLIT>(j).
template <int T>
struct Raw8 {
    uint4 v[T == kF32 ? 2 : 1];
};

template <bool SPLIT>
__device__ __forceinline__ constexpr int at8(int j) {
    return SPLIT && j >= 4 ? j + 124 : j;
}

// First index of the i-th eight of a thread, in a row that `threads` share
// (a multiple of 32).
template <bool SPLIT>
__device__ __forceinline__ int64_t first8(unsigned thread, unsigned i, unsigned threads) {
    const int64_t t = static_cast<int64_t>(i) * threads + thread;
    return SPLIT ? 8 * (t & ~static_cast<int64_t>(31)) + 4 * (thread & 31) : 8 * t;
}

// Four elements from p on, the first n of them valid, as words (fp32: four,
// bf16: two); the others are zero, without touching memory.
template <int T>
__device__ __forceinline__ void load_raw4(const uint8_t *p, int64_t n, uint32_t *w) {
    if (n >= 4) {
        if constexpr (T == kF32) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < (T == kF32 ? 4 : 2); ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (i < n) {
            if constexpr (T == kF32) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
            else w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << (16 * (i & 1));
        }
    }
}

// The eight elements at e, those at K and beyond as zero.  Rows are 16-byte
// aligned and groups start at multiples of four (SPLIT) or eight, so a whole
// group is one aligned access.
template <int T, bool SPLIT>
__device__ __forceinline__ Raw8<T> load_raw8(const void *row, int64_t e, int64_t K) {
    Raw8<T> r;
    const uint8_t *p = static_cast<const uint8_t *>(row) + e * elem_bytes<T>;
    if constexpr (T == kBF16 && !SPLIT) {
        if (e + 8 <= K) {
            r.v[0] = *reinterpret_cast<const uint4 *>(p);
            return r;
        }
    }
    uint32_t w[T == kF32 ? 8 : 4];
    load_raw4<T>(p, K - e, w);
    load_raw4<T>(p + at8<SPLIT>(4) * elem_bytes<T>, K - e - at8<SPLIT>(4), w + (T == kF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (T == kF32 ? 2 : 1); ++i)
        r.v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    return r;
}

template <int T>
__device__ __forceinline__ void widen8(const Raw8<T> &r, float (&f)[8]) {
    if constexpr (T == kF32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i] = __uint_as_float(r.v[i].x);
            f[4 * i + 1] = __uint_as_float(r.v[i].y);
            f[4 * i + 2] = __uint_as_float(r.v[i].z);
            f[4 * i + 3] = __uint_as_float(r.v[i].w);
        }
    } else {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // a bf16 is the upper half of its fp32
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

template <int T, bool SPLIT>
__device__ __forceinline__ void load8(const void *row, int64_t e, int64_t K, float (&f)[8]) {
    widen8<T>(load_raw8<T, SPLIT>(row, e, K), f);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

template <int T>
__device__ __forceinline__ void store4(uint8_t *p, int64_t n, const float *f) {
    if (n >= 4) {
        if constexpr (T == kF32) *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        else *reinterpret_cast<uint2 *>(p) = make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]));
        return;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (i < n) {
            if constexpr (T == kF32) reinterpret_cast<float *>(p)[i] = f[i];
            else reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(f[i]);
        }
    }
}

// Writes the eight elements at e, rounded to T (nearest even); those at K and
// beyond are not written.
template <int T, bool SPLIT>
__device__ __forceinline__ void store8(void *row, int64_t e, int64_t K, const float (&f)[8]) {
    uint8_t *p = static_cast<uint8_t *>(row) + e * elem_bytes<T>;
    if constexpr (T == kBF16 && !SPLIT) {
        if (e + 8 <= K) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]),
                                                       bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
            return;
        }
    }
    store4<T>(p, K - e, &f[0]);
    store4<T>(p + at8<SPLIT>(4) * elem_bytes<T>, K - e - at8<SPLIT>(4), &f[4]);
}

// The values as they will read back once stored as T.
template <int T>
__device__ __forceinline__ void round8(float (&f)[8]) {
    if constexpr (T == kBF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __bfloat162float(__float2bfloat16_rn(f[i]));
    }
}

// Start of every kernel here (launched with programmatic dependence, so that
// its blocks may take their places while the kernel before it in the stream
// still runs): nothing is read or written before that kernel has finished
// and its writes are visible; then the next one's blocks may come.
__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
    return v;
}

// ------------------------------------------------------------------ MXFP8 --
//
// A block is 32 consecutive values along K.  Its scale is the smallest power
// of two 2^e, e in [-127, 127], with |v| <= 448 * 2^e for every finite v of the
// block (448 is E4M3's largest value), so no finite value saturates; a code
// is v / 2^e rounded to nearest even.  NaN and infinities get E4M3's NaN code
// 0x7F and do not count for the scale (E4M3 has no infinity).

// Largest finite |v| of N values.  Infinities become NaN on the way, which the
// maximum passes over and the conversion turns into the NaN code; testing for
// them once per N values keeps the common path at one instruction a value.
template <int N>
__device__ __forceinline__ float finite_max(float *v) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]));
    if (m == __uint_as_float(0x7F800000u)) {
        m = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (fabsf(v[i]) == __uint_as_float(0x7F800000u)) v[i] = __uint_as_float(0x7FC00000u);
            m = fmaxf(m, fabsf(v[i]));
        }
    }
    return m;
}

// The E8M0 byte (e + 127) for a block whose largest magnitude is amax = 1.f *
// 2^(E-127): with 448 = 1.75 * 2^8, e = E - 127 - 8, one more where 1.f > 1.75.
// Blocks of zeros and of values below 448 * 2^-127 get byte 0.
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int b = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(max(b, 0));
}

// 2^-e for an E8M0 byte e + 127 <= 247: always a normal fp32.
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Two codes: the values times 2^-e (exact, or far below the smallest code),
// rounded; a NaN gives 0x7F.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi, float inv) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi * inv), "f"(lo * inv));
    return d;
}

__device__ __forceinline__ uint32_t e4m3_codes4(const float *v, float inv) {
    return e4m3_pair(v[0], v[1], inv) | (e4m3_pair(v[2], v[3], inv) << 16);
}

// Encodes the eights of a warp (the values at e of each lane, K a multiple of
// 32): a block of 32 is four lanes' eights, or with SPLIT eight lanes' fours.
// All 32 lanes call it, those past K with zeros.  q, sf: the row's codes
// and scales.
template <bool SPLIT>
__device__ __forceinline__ void mx_store8(float (&v)[8], int64_t e, int64_t K, uint8_t *q, uint8_t *sf) {
    if constexpr (SPLIT) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float m = finite_max<4>(&v[4 * h]);
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
            const int64_t eh = e + 128 * h;
            if (eh < K) {
                const uint32_t byte = mx_scale_byte(m);
                *reinterpret_cast<uint32_t *>(q + eh) = e4m3_codes4(&v[4 * h], mx_inv_scale(byte));
                if ((threadIdx.x & 7) == 0) sf[eh / 32] = static_cast<uint8_t>(byte);
            }
        }
    } else {
        float m = finite_max<8>(v);
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        if (e < K) {
            const uint32_t byte = mx_scale_byte(m);
            const float inv = mx_inv_scale(byte);
            *reinterpret_cast<uint2 *>(q + e) = make_uint2(e4m3_codes4(&v[0], inv), e4m3_codes4(&v[4], inv));
            if ((threadIdx.x & 3) == 0) sf[e / 32] = static_cast<uint8_t>(byte);
        }
    }
}

}  // namespace b200
