// RMS norm with the residual's addition, forward and backward.
//
//   h = x + r (rounded to h's type),  rstd = 1 / sqrt(mean(h^2) + eps),
//   y = h * rstd * w
// and with g = dy * w, n = h * rstd:
//   dh = rstd * (g - n * mean(g * n)) (+ dr),   dw = sum over rows of dy * n.
//
// Both are bound by memory: a row is read once, stays in registers between
// the sum over it and its use, and is written once.  A row belongs to
// blockDim.x threads (a multiple of 32), thread t holding the vectors t,
// t + blockDim.x, ... of eight elements; short rows take one warp each, and
// blockDim.y of them share a block.  All sums are fp32, in a fixed order.
#pragma once
#include "rows.cuh"

namespace b200 {

// Sum over the threads of a row.  With more than one warp per row the block
// holds one row only; `red` has two halves that alternate by `phase`, so that
// one barrier per sum is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float (*red)[N][32], int phase) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = warp_sum(s[i]);
    if (blockDim.x == 32) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) red[phase][i][warp] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = warp_sum(lane < warps ? red[phase][i][lane] : 0.0f);
}

struct RmsnormArgs {
    const void *x, *r;
    void *h;
    const float *w;
    void *y;
    uint8_t *q, *sf;
    float *rstd;
    int64_t M, K, ldx, ldr, ldh, ldy, ldq;
    float eps;
};

__device__ __forceinline__ void rmsnorm_write(const RmsnormArgs &a, int64_t row, int64_t e, const float (&h)[8],
                                              const float (&w)[8], float rstd) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = h[i] * rstd * w[i];
    if (a.y) store8<kBF16>(static_cast<__nv_bfloat16 *>(a.y) + row * a.ldy, e, a.K - e, y);
    if (a.q) mx_store8(y, e < a.K, a.q + row * a.ldq + e, a.sf + row * (a.K / 32) + e / 32);
}

// One row in registers: VPT vectors per thread.
template <int XT, int HT, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) rmsnorm_kernel(RmsnormArgs a) {
    __shared__ float red[2][1][32];
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.M) return;   // whole warps, and only where a row has one warp
    const uint8_t *x = static_cast<const uint8_t *>(a.x) + row * a.ldx * elem_bytes<XT>;
    float v[VPT][8], w[8];
    {
        Raw8<XT> rx[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int64_t e = 8 * (static_cast<int64_t>(threadIdx.x) + static_cast<int64_t>(i) * blockDim.x);
            rx[i] = load_raw8<XT>(x, e, a.K - e);
        }
        if constexpr (HT != kNone) {
            const uint8_t *r = static_cast<const uint8_t *>(a.r) + row * a.ldr * elem_bytes<HT>;
            uint8_t *h = static_cast<uint8_t *>(a.h) + row * a.ldh * elem_bytes<HT>;
            Raw8<HT> rr[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t e = 8 * (static_cast<int64_t>(threadIdx.x) + static_cast<int64_t>(i) * blockDim.x);
                rr[i] = load_raw8<HT>(r, e, a.K - e);
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t e = 8 * (static_cast<int64_t>(threadIdx.x) + static_cast<int64_t>(i) * blockDim.x);
                float f[8];
                widen8<XT>(rx[i], v[i]);
                widen8<HT>(rr[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += f[j];
                round8<HT>(v[i]);   // the norm is of the sum as it is stored
                if (a.h) store8<HT>(h, e, a.K - e, v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) widen8<XT>(rx[i], v[i]);
        }
    }
    // with one vector per thread (few rows) the weights' latency overlaps the sum
    if constexpr (VPT == 1) load8<kF32>(a.w, 8 * static_cast<int64_t>(threadIdx.x), a.K - 8 * static_cast<int64_t>(threadIdx.x), w);
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += v[i][j] * v[i][j];
    row_sum<1>(s, red, 0);
    const float rstd = 1.0f / sqrtf(s[0] / static_cast<float>(a.K) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t e = 8 * (static_cast<int64_t>(threadIdx.x) + static_cast<int64_t>(i) * blockDim.x);
        if constexpr (VPT > 1) load8<kF32>(a.w, e, a.K - e, w);
        rmsnorm_write(a, row, e, v[i], w, rstd);
    }
}

// Rows too long for registers: a second pass reads them again (from L2, where
// they fit).  It reads h where h was stored (r may be the same buffer, and
// then holds h by now: each thread reads back what it wrote itself).
template <int XT, int HT>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(RmsnormArgs a) {
    __shared__ float red[2][1][32];
    const int64_t row = blockIdx.x;
    const uint8_t *x = static_cast<const uint8_t *>(a.x) + row * a.ldx * elem_bytes<XT>;
    const uint8_t *r = static_cast<const uint8_t *>(a.r) + row * a.ldr * elem_bytes<HT>;
    uint8_t *h = static_cast<uint8_t *>(a.h) + row * a.ldh * elem_bytes<HT>;
    const int64_t step = 8 * static_cast<int64_t>(blockDim.x);
    auto sum_of = [&](int64_t e, float (&v)[8]) {
        load8<XT>(x, e, a.K - e, v);
        if constexpr (HT != kNone) {
            float f[8];
            load8<HT>(r, e, a.K - e, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += f[j];
            round8<HT>(v);
        }
    };
    float s[1] = {0.0f};
    for (int64_t e = 8 * static_cast<int64_t>(threadIdx.x); e < a.K; e += step) {
        float v[8];
        sum_of(e, v);
        if constexpr (HT != kNone) {
            if (a.h) store8<HT>(h, e, a.K - e, v);
        }
        float p = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) p += v[j] * v[j];
        s[0] += p;
    }
    row_sum<1>(s, red, 0);
    const float rstd = 1.0f / sqrtf(s[0] / static_cast<float>(a.K) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    // every thread of a warp stays in the loop (the codes' maximum is taken across lanes)
    for (int64_t e0 = 0; e0 < a.K; e0 += step) {
        const int64_t e = e0 + 8 * static_cast<int64_t>(threadIdx.x);
        float v[8], w[8];
        if (HT != kNone && a.h) load8<HT == kNone ? kF32 : HT>(h, e, a.K - e, v);
        else sum_of(e, v);
        load8<kF32>(a.w, e, a.K - e, w);
        rmsnorm_write(a, row, e, v, w, rstd);
    }
}

// --------------------------------------------------------------- backward --

struct RmsnormBackArgs {
    const void *dy, *h;
    const float *w, *rstd;
    const void *dr;
    void *dh;
    float *partial;   // [gridDim.x][K]: this block's share of dw; null: no dw
    int64_t M, K, lddy, ldh, lddr, lddh;
};

// Persistent blocks: block b takes rows b, b + gridDim.x, ... (times
// blockDim.y) and keeps its share of dw in registers, written out once at
// the end and summed over the blocks by rmsnorm_dw_kernel in block order.
template <int YT, int HT, int DT, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) rmsnorm_back_kernel(RmsnormBackArgs a) {
    __shared__ float red[2][1][32];
    float dw[VPT][8] = {};
    int phase = 0;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.M; row += stride) {
        const uint8_t *dy = static_cast<const uint8_t *>(a.dy) + row * a.lddy * elem_bytes<YT>;
        const uint8_t *h = static_cast<const uint8_t *>(a.h) + row * a.ldh * elem_bytes<HT>;
        const uint8_t *dr = static_cast<const uint8_t *>(a.dr) + row * a.lddr * elem_bytes<DT>;
        uint8_t *dh = static_cast<uint8_t *>(a.dh) + row * a.lddh * elem_bytes<DT>;
        const float rstd = a.rstd[row];
        Raw8<YT> ry[VPT];
        Raw8<HT> rh[VPT];
        Raw8<DT> rr[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int64_t e = 8 * (static_cast<int64_t>(threadIdx.x) + static_cast<int64_t>(i) * blockDim.x);
            ry[i] = load_raw8<YT>(dy, e, a.K - e);
            rh[i] = load_raw8<HT>(h, e, a.K - e);
        }
        if (a.dr) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int64_t e = 8 * (static_cast<int64_t>(threadIdx.x) + static_cast<int64_t>(i) * blockDim.x);
                rr[i] = load_raw8<DT>(dr, e, a.K - e);
            }
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int64_t e = 8 * (static_cast<int64_t>(threadIdx.x) + static_cast<int64_t>(i) * blockDim.x);
            float y[8], v[8], w[8];
            widen8<YT>(ry[i], y);
            widen8<HT>(rh[i], v);
            load8<kF32>(a.w, e, a.K - e, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = v[j] * rstd;
                s[0] += y[j] * w[j] * n;
                dw[i][j] += y[j] * n;
            }
        }
        row_sum<1>(s, red, phase);
        phase ^= 1;
        const float mean = s[0] / static_cast<float>(a.K);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int64_t e = 8 * (static_cast<int64_t>(threadIdx.x) + static_cast<int64_t>(i) * blockDim.x);
            float y[8], v[8], w[8], d[8];
            widen8<YT>(ry[i], y);
            widen8<HT>(rh[i], v);
            load8<kF32>(a.w, e, a.K - e, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = rstd * (y[j] * w[j] - v[j] * rstd * mean);
            if (a.dr) {
                float f[8];
                widen8<DT>(rr[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] += f[j];
            }
            store8<DT>(dh, e, a.K - e, d);
        }
    }
    if (!a.partial) return;
    // the rows of one block (short rows: one warp each) in threadIdx.y order
    extern __shared__ float acc[];
    if (blockDim.y > 1) {
        for (unsigned r = 0; r < blockDim.y; ++r) {
            if (threadIdx.y == r) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float *p = &acc[(i * 8 + j) * 32 + threadIdx.x];
                        *p = r ? *p + dw[i][j] : dw[i][j];
                    }
            }
            __syncthreads();
        }
        if (threadIdx.y != 0) return;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) dw[i][j] = acc[(i * 8 + j) * 32 + threadIdx.x];
    }
    // rows of `partial` are K floats apart, which need not keep 16-byte alignment
    float *p = a.partial + static_cast<int64_t>(blockIdx.x) * a.K;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t e = 8 * (static_cast<int64_t>(threadIdx.x) + static_cast<int64_t>(i) * blockDim.x);
        if ((a.K & 3) == 0) {
            store8<kF32>(p, e, a.K - e, dw[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e + j < a.K) p[e + j] = dw[i][j];
        }
    }
}

// Rows too long for registers: two passes over each row, and the block's share
// of dw kept in `partial` itself (each thread owns its columns there).
template <int YT, int HT, int DT>
__global__ void __launch_bounds__(1024) rmsnorm_back_long_kernel(RmsnormBackArgs a) {
    __shared__ float red[2][1][32];
    int phase = 0;
    const int64_t step = 8 * static_cast<int64_t>(blockDim.x);
    bool first = true;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, first = false) {
        const uint8_t *dy = static_cast<const uint8_t *>(a.dy) + row * a.lddy * elem_bytes<YT>;
        const uint8_t *h = static_cast<const uint8_t *>(a.h) + row * a.ldh * elem_bytes<HT>;
        const uint8_t *dr = static_cast<const uint8_t *>(a.dr) + row * a.lddr * elem_bytes<DT>;
        uint8_t *dh = static_cast<uint8_t *>(a.dh) + row * a.lddh * elem_bytes<DT>;
        const float rstd = a.rstd[row];
        float s[1] = {0.0f};
        for (int64_t e = 8 * static_cast<int64_t>(threadIdx.x); e < a.K; e += step) {
            float y[8], v[8], w[8], p = 0.0f;
            load8<YT>(dy, e, a.K - e, y);
            load8<HT>(h, e, a.K - e, v);
            load8<kF32>(a.w, e, a.K - e, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) p += y[j] * w[j] * (v[j] * rstd);
            s[0] += p;
        }
        row_sum<1>(s, red, phase);
        phase ^= 1;
        const float mean = s[0] / static_cast<float>(a.K);
        for (int64_t e = 8 * static_cast<int64_t>(threadIdx.x); e < a.K; e += step) {
            float y[8], v[8], w[8], d[8];
            load8<YT>(dy, e, a.K - e, y);
            load8<HT>(h, e, a.K - e, v);
            load8<kF32>(a.w, e, a.K - e, w);
            if (a.dr) load8<DT>(dr, e, a.K - e, d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = v[j] * rstd;
                const float g = rstd * (y[j] * w[j] - n * mean);
                d[j] = a.dr ? g + d[j] : g;
                if (a.partial && e + j < a.K) {
                    float *p = a.partial + static_cast<int64_t>(blockIdx.x) * a.K + e + j;
                    *p = first ? y[j] * n : *p + y[j] * n;
                }
            }
            store8<DT>(dh, e, a.K - e, d);
        }
    }
}

// dw[k] = sum over the blocks' shares, in block order within each of the 8
// warps of a block and then over the warps: 32 columns per block.
__global__ void __launch_bounds__(256) rmsnorm_dw_kernel(const float *__restrict__ partial, float *dw, int64_t rows,
                                                         int64_t K) {
    __shared__ float part[8][32];
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;
    const int warp = threadIdx.x / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.0f;
    if (col < K) {
#pragma unroll 4
        for (int64_t r = warp; r < rows; r += 8) s += __ldcg(&partial[r * K + col]);
    }
    part[warp][threadIdx.x % 32] = s;
    __syncthreads();
    if (warp == 0 && col < K) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[i][threadIdx.x];
        dw[col] = s;
    }
}

}  // namespace b200
