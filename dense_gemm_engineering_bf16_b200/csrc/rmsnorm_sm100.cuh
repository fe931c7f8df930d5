// RMS norm with the residual's addition, forward and backward.
//
//   h = x + r (rounded to h's type),  rstd = 1 / sqrt(mean(h^2) + eps),
//   y = h * rstd * w
// and with g = dy * w, n = h * rstd:
//   dh = rstd * (g - n * mean(g * n)) (+ dr),   dw = sum over rows of dy * n.
//
// Both are bound by memory: a row is read once, stays in registers between
// the sum over it and its use, and is written once.  A row belongs to
// blockDim.x threads (a multiple of 32), each holding one or more eights of
// elements; blockDim.y short rows share a block (one warp each in the forward
// pass).  All sums are fp32, in a fixed order.
#pragma once
#include "rows.cuh"

namespace b200 {

// Sum over the blockDim.x threads of a row.  With more than one warp per row
// the warps of a row meet at a barrier of their own (1 + threadIdx.y, at most
// 8: rows of two warps are up to eight to a block), and `red`, their row's, has
// two halves that alternate by `phase`, so that one barrier per sum is enough.
// SHARED: several rows of more than one warp may share the block.
constexpr int kMaxRows = 16;

template <bool SHARED>
__device__ __forceinline__ float row_sum(float s, float (*red)[32], int phase) {
    s = warp_sum(s);
    if (blockDim.x == 32) return s;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (lane == 0) red[phase][warp] = s;
    if constexpr (SHARED) asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
    else __syncthreads();
    return warp_sum(lane < warps ? red[phase][lane] : 0.0f);
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

template <bool SPLIT>
__device__ __forceinline__ void rmsnorm_write(const RmsnormArgs &a, int64_t row, int64_t e, const float (&h)[8],
                                              const float (&w)[8], float rstd) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = h[i] * rstd * w[i];
    if (a.y) store8<kBF16, SPLIT>(static_cast<__nv_bfloat16 *>(a.y) + row * a.ldy, e, a.K, y);
    if (a.q) mx_store8<SPLIT>(y, e, a.K, a.q + row * a.ldq, a.sf + row * (a.K / 32));
}

// One row in registers: VPT eights per thread.  8192 x 8192 with a bf16 residual,
// codes out: 75.3 us, 96 % of the copy rate; 4000 x 3000 with an fp32 stream: 24.3
// us, 90 %; one row of 8192: 2.6 us, all of it launch and two trips to memory.
template <int XT, int HT, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) rmsnorm_kernel(RmsnormArgs a) {
    constexpr bool SPLIT = XT == kF32 || HT == kF32;
    __shared__ float red[2][32];
    wait_for_stream();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.M) return;   // whole warps, and only where a row has one warp
    const uint8_t *x = static_cast<const uint8_t *>(a.x) + row * a.ldx * elem_bytes<XT>;
    float v[VPT][8], w[8];
    {
        Raw8<XT> rx[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            rx[i] = load_raw8<XT, SPLIT>(x, first8<SPLIT>(threadIdx.x, i, blockDim.x), a.K);
        if constexpr (HT != kNone) {
            const uint8_t *r = static_cast<const uint8_t *>(a.r) + row * a.ldr * elem_bytes<HT>;
            uint8_t *h = static_cast<uint8_t *>(a.h) + row * a.ldh * elem_bytes<HT>;
            Raw8<HT> rr[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                rr[i] = load_raw8<HT, SPLIT>(r, first8<SPLIT>(threadIdx.x, i, blockDim.x), a.K);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float f[8];
                widen8<XT>(rx[i], v[i]);
                widen8<HT>(rr[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += f[j];
                round8<HT>(v[i]);   // the norm is of the sum as it is stored
                if (a.h) store8<HT, SPLIT>(h, first8<SPLIT>(threadIdx.x, i, blockDim.x), a.K, v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) widen8<XT>(rx[i], v[i]);
        }
    }
    // with one eight per thread (few rows) the weights' latency overlaps the sum
    if constexpr (VPT == 1) load8<kF32, SPLIT>(a.w, first8<SPLIT>(threadIdx.x, 0, blockDim.x), a.K, w);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[i][j] * v[i][j];
    s = row_sum<false>(s, red, 0);
    const float rstd = 1.0f / sqrtf(s / static_cast<float>(a.K) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int64_t e = first8<SPLIT>(threadIdx.x, i, blockDim.x);
        if constexpr (VPT > 1) load8<kF32, SPLIT>(a.w, e, a.K, w);
        rmsnorm_write<SPLIT>(a, row, e, v[i], w, rstd);
    }
}

// Rows too long for registers (past 16384 elements): a second pass reads them
// again (from L2, where they fit; 2000 x 20000 bf16 with a residual: 68.8 us, 71 % of
// the copy rate).  It reads h where h was stored (r may be the same buffer, and
// then holds h by now: each thread reads back what it wrote itself).
template <int XT, int HT>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(RmsnormArgs a) {
    constexpr bool SPLIT = XT == kF32 || HT == kF32;
    __shared__ float red[2][32];
    wait_for_stream();
    const int64_t row = blockIdx.x;
    const uint8_t *x = static_cast<const uint8_t *>(a.x) + row * a.ldx * elem_bytes<XT>;
    const uint8_t *r = static_cast<const uint8_t *>(a.r) + row * a.ldr * elem_bytes<HT>;
    uint8_t *h = static_cast<uint8_t *>(a.h) + row * a.ldh * elem_bytes<HT>;
    const int64_t steps = (a.K + 8191) / 8192;
    auto sum_of = [&](int64_t e, float (&v)[8]) {
        load8<XT, SPLIT>(x, e, a.K, v);
        if constexpr (HT != kNone) {
            float f[8];
            load8<HT, SPLIT>(r, e, a.K, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += f[j];
            round8<HT>(v);
        }
    };
    float s = 0.0f;
    for (int64_t i = 0; i < steps; ++i) {
        const int64_t e = 8192 * i + first8<SPLIT>(threadIdx.x, 0, 1024);
        float v[8];
        sum_of(e, v);
        if constexpr (HT != kNone) {
            if (a.h) store8<HT, SPLIT>(h, e, a.K, v);
        }
        float p = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) p += v[j] * v[j];
        s += p;
    }
    s = row_sum<false>(s, red, 0);
    const float rstd = 1.0f / sqrtf(s / static_cast<float>(a.K) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    for (int64_t i = 0; i < steps; ++i) {
        const int64_t e = 8192 * i + first8<SPLIT>(threadIdx.x, 0, 1024);
        float v[8], w[8];
        if (HT != kNone && a.h) load8<HT == kNone ? kF32 : HT, SPLIT>(h, e, a.K, v);
        else sum_of(e, v);
        load8<kF32, SPLIT>(a.w, e, a.K, w);
        rmsnorm_write<SPLIT>(a, row, e, v, w, rstd);
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
    int ring;         // rows in shared memory at a time: 2, 3 or 4
    float inv_k;      // 1 / K
    bool stage_dr;    // dr goes through shared memory too
};

// This thread's eight elements at e into shared memory, asynchronously, the
// row's end included (a thread that waited for its few last elements there
// would hold up the whole block once per row).  Copied by the thread that
// reads them back, so that no barrier stands between.  What lies at K and
// beyond stays as it is in the slot.
template <int BYTES>
__device__ __forceinline__ void stage_copy(uint8_t *dst, const uint8_t *src) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else if constexpr (BYTES == 2)      // two bytes read, two more zero
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, 2;" ::"r"(d), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
}

template <int T>
__device__ __forceinline__ void stage4(uint8_t *dst, const uint8_t *src, int n) {
    if (n >= 4) {
        stage_copy<4 * elem_bytes<T>>(dst, src);
        return;
    }
#pragma unroll
    for (int i = 0; i < 3; i += 4 / elem_bytes<T>) {
        if (i + 4 / elem_bytes<T> <= n) stage_copy<4>(dst + i * elem_bytes<T>, src + i * elem_bytes<T>);
        else if (i < n) stage_copy<2>(dst + i * elem_bytes<T>, src + i * elem_bytes<T>);
    }
}

template <int T, bool SPLIT>
__device__ __forceinline__ void stage8(uint8_t *slot, unsigned pitch, const uint8_t *row, int e, int K) {
    const uint8_t *p = row + e * elem_bytes<T>;
    if constexpr (T == kBF16 && !SPLIT) {
        if (e + 8 <= K) {
            stage_copy<16>(slot, p);
            return;
        }
    }
    stage4<T>(slot, p, K - e);
    stage4<T>(slot + (T == kF32 ? pitch : 8), p + at8<SPLIT>(4) * elem_bytes<T>, K - e - at8<SPLIT>(4));
}

template <int T>
__device__ __forceinline__ void staged8(const uint8_t *slot, unsigned pitch, float (&f)[8]) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (T == kF32 ? 2 : 1); ++i) r.v[i] = *reinterpret_cast<const uint4 *>(slot + i * pitch);
    widen8<T>(r, f);
}

// 16-byte pieces per eight of what is staged: dy, h, and dr where two rows with
// it fit into shared memory (else dr is read when it is needed).
template <int YT, int HT, int DT>
constexpr int back_pieces(bool stage_dr) {
    return (YT == kF32 ? 2 : 1) + (HT == kF32 ? 2 : 1) + (!stage_dr ? 0 : DT == kF32 ? 2 : 1);
}

// Persistent blocks: block b takes rows b, b + gridDim.x, ... (times
// blockDim.y) and keeps its share of dw in registers, written out once at
// the end and summed over the blocks by rmsnorm_dw_kernel in block order.
// Short rows share a block of 512 threads, each with a barrier of its own.
// The next rows are on their way into shared memory while one is summed and
// written (the barrier in the middle of each row would leave memory idle
// otherwise), and what a row's second half needs is read from there again,
// which keeps registers free.  With a residual's gradient: 8192 x 8192 bf16 97.5
// us, 84 % of the copy rate (a barrier and ten shuffles per row are what is left,
// with one block of 16 warps per SM); 4000 x 3000 fp32 33.5 us, 77 %; with four
// eights per thread, two rows in shared memory and 96 to 128 registers, 2000 x
// 16384 bf16 63 us, 63 %, and 2000 x 12000 fp32 89 us, 66 %.  1000 x 2000 bf16
// without one: 8.3 us, two launches and seven rows per block.
template <int YT, int HT, int DT, int VPT>
__global__ void __launch_bounds__(512) rmsnorm_back_kernel(RmsnormBackArgs a) {
    constexpr bool SPLIT = YT == kF32 || HT == kF32 || DT == kF32;
    // four eights per thread only where a row needs more than 256 threads
    constexpr bool SHARED = VPT < 4;
    __shared__ float red[SHARED ? kMaxRows : 1][2][32];
    wait_for_stream();
    const unsigned sub = SHARED ? threadIdx.y : 0, subs = SHARED ? blockDim.y : 1;   // row of the block
    extern __shared__ __align__(16) uint8_t dyn[];
    constexpr int kY = YT == kF32 ? 2 : 1, kH = HT == kF32 ? 2 : 1, kD = DT == kF32 ? 2 : 1;
    const bool stage_dr = VPT < 4 || a.stage_dr;
    const int pieces = kY + kH + (stage_dr ? kD : 0);
    const unsigned pitch = 16 * blockDim.x * subs;             // between a thread's pieces
    const unsigned row_pitch = VPT * pieces * pitch, ring_end = a.ring * row_pitch;
    uint8_t *const mine = dyn + 16 * (sub * blockDim.x + threadIdx.x);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * subs;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * subs + sub;
    const int K = static_cast<int>(a.K);                       // at most 16384 here
    unsigned fill = 0;
    // the next row to load, and this thread's first vector of it
    const int e0 = static_cast<int>(first8<SPLIT>(threadIdx.x, 0, blockDim.x));
    int64_t ahead = first;
    const uint8_t *dy = static_cast<const uint8_t *>(a.dy) + first * a.lddy * elem_bytes<YT>;
    const uint8_t *h = static_cast<const uint8_t *>(a.h) + first * a.ldh * elem_bytes<HT>;
    const uint8_t *dr = static_cast<const uint8_t *>(a.dr) + first * a.lddr * elem_bytes<DT>;
    const int64_t dy_step = stride * a.lddy * elem_bytes<YT>, h_step = stride * a.ldh * elem_bytes<HT>;
    const int64_t dr_step = stride * a.lddr * elem_bytes<DT>;
    auto load_row = [&]() {
        if (ahead < a.M) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int e = e0 + 8 * i * static_cast<int>(blockDim.x);
                if (e >= K) break;
                uint8_t *p = mine + fill + i * pieces * pitch;
                stage8<YT, SPLIT>(p, pitch, dy, e, K);
                stage8<HT, SPLIT>(p + kY * pitch, pitch, h, e, K);
                if (stage_dr && a.dr) stage8<DT, SPLIT>(p + (kY + kH) * pitch, pitch, dr, e, K);
            }
        }
        ahead += stride;
        dy += dy_step;
        h += h_step;
        dr += dr_step;
        fill = fill + row_pitch == ring_end ? 0 : fill + row_pitch;
        asm volatile("cp.async.commit_group;" ::: "memory");   // one group per row, empty ones too
    };
    // elements past K read as zero from every slot: they add nothing to any sum
    for (int r = 0; r < a.ring; ++r)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (e0 + 8 * i * static_cast<int>(blockDim.x) + at8<SPLIT>(7) >= K)
                for (int q = 0; q < pieces; ++q)
                    *reinterpret_cast<uint4 *>(mine + r * row_pitch + (i * pieces + q) * pitch) =
                        make_uint4(0, 0, 0, 0);
    for (int i = 1; i < a.ring; ++i) load_row();

    float dw[VPT][8] = {}, w[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) load8<kF32, SPLIT>(a.w, e0 + 8 * i * static_cast<int>(blockDim.x), K, w[i]);
    float rstd = first < a.M ? a.rstd[first] : 0.0f;
    uint8_t *dh = static_cast<uint8_t *>(a.dh) + first * a.lddh * elem_bytes<DT>;
    int phase = 0;
    unsigned slot = 0;
    for (int64_t row = first; row < a.M; row += stride) {
        if (a.ring == 4) asm volatile("cp.async.wait_group 2;" ::: "memory");
        else if (a.ring == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        load_row();     // into the slot this thread read in the previous iteration
        const float next_rstd = row + stride < a.M ? a.rstd[row + stride] : 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint8_t *p = mine + slot + i * pieces * pitch;
            float y[8], v[8];
            staged8<YT>(p, pitch, y);
            staged8<HT>(p + kY * pitch, pitch, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // n first: dy h may leave fp32's range where dy n does not
                const float p = y[j] * (v[j] * rstd);
                dw[i][j] += p;
                s += p * w[i][j];
            }
        }
        s = row_sum<SHARED>(s, red[sub], phase);
        phase ^= 1;
        // n mean(g n) = h c with c = rstd mean(g n): no rstd^2, which passes fp32's
        // range in a row of zeros with a subnormal eps
        const float c = rstd * (s * a.inv_k);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int e = e0 + 8 * i * static_cast<int>(blockDim.x);
            const uint8_t *p = mine + slot + i * pieces * pitch;
            float y[8], v[8], d[8];
            staged8<YT>(p, pitch, y);
            staged8<HT>(p + kY * pitch, pitch, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = y[j] * w[i][j] - v[j] * c;
            if (a.dr) {
                float f[8];
                if (stage_dr)
                    staged8<DT>(p + (kY + kH) * pitch, pitch, f);
                else
                    load8<DT, SPLIT>(static_cast<const uint8_t *>(a.dr) + row * a.lddr * elem_bytes<DT>, e, K, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = rstd * d[j] + f[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] *= rstd;
            }
            store8<DT, SPLIT>(dh, e, K, d);
        }
        rstd = next_rstd;
        dh += stride * a.lddh * elem_bytes<DT>;
        slot = slot + row_pitch == ring_end ? 0 : slot + row_pitch;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.partial) return;
    // the sums of a block's rows meet in shared memory and are added in the rows' order
    if (SHARED && subs > 1) {
        const int T = static_cast<int>(blockDim.x), sums = VPT * 8 * T, threads = T * static_cast<int>(subs);
        float *acc = reinterpret_cast<float *>(dyn);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int at = sub * sums + 8 * (i * T + static_cast<int>(threadIdx.x));
            float4 *d = reinterpret_cast<float4 *>(acc + at);
            d[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            d[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
        __syncthreads();
        for (int at = static_cast<int>(sub) * T + static_cast<int>(threadIdx.x); at < sums; at += threads) {
            float v = 0.0f;
            for (unsigned r = 0; r < subs; ++r) v += acc[r * sums + at];
            const int64_t col = first8<SPLIT>(at / 8, 0, T) + at8<SPLIT>(at % 8);
            if (col < K) a.partial[static_cast<int64_t>(blockIdx.x) * a.K + col] = v;
        }
        return;
    }
    // rows of `partial` are K floats apart: 16-byte aligned where K is a multiple of four
    float *p = a.partial + static_cast<int64_t>(blockIdx.x) * a.K;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int e = e0 + 8 * i * static_cast<int>(blockDim.x);
        if ((K & 3) == 0) {
            store8<kF32, SPLIT>(p, e, K, dw[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e + at8<SPLIT>(j) < K) p[e + at8<SPLIT>(j)] = dw[i][j];
        }
    }
}

// Rows of which shared memory does not hold two (from 13313 elements on with dy
// and h both fp32) or registers one (past 16384): two passes over each row, and the
// block's share of dw kept in `partial` itself (each thread owns its columns
// there), read and written once per row, which is what bounds it: with a
// residual's gradient 2000 x 13320 fp32 150 us, 43 % of the copy rate (at 13312, on the
// kernel above, 92 us), 2000 x 20000 bf16 255 us, 19 %.
template <int YT, int HT, int DT>
__global__ void __launch_bounds__(1024) rmsnorm_back_long_kernel(RmsnormBackArgs a) {
    constexpr bool SPLIT = YT == kF32 || HT == kF32 || DT == kF32;
    __shared__ float red[2][32];
    wait_for_stream();
    int phase = 0;
    const int64_t steps = (a.K + 8191) / 8192;
    bool first = true;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, first = false) {
        const uint8_t *dy = static_cast<const uint8_t *>(a.dy) + row * a.lddy * elem_bytes<YT>;
        const uint8_t *h = static_cast<const uint8_t *>(a.h) + row * a.ldh * elem_bytes<HT>;
        const uint8_t *dr = static_cast<const uint8_t *>(a.dr) + row * a.lddr * elem_bytes<DT>;
        uint8_t *dh = static_cast<uint8_t *>(a.dh) + row * a.lddh * elem_bytes<DT>;
        const float rstd = a.rstd[row];
        float s = 0.0f;
        for (int64_t i = 0; i < steps; ++i) {
            const int64_t e = 8192 * i + first8<SPLIT>(threadIdx.x, 0, 1024);
            float y[8], v[8], w[8], p = 0.0f;
            load8<YT, SPLIT>(dy, e, a.K, y);
            load8<HT, SPLIT>(h, e, a.K, v);
            load8<kF32, SPLIT>(a.w, e, a.K, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) p += y[j] * w[j] * (v[j] * rstd);
            s += p;
        }
        s = row_sum<false>(s, red, phase);
        phase ^= 1;
        const float mean = s / static_cast<float>(a.K);
        for (int64_t i = 0; i < steps; ++i) {
            const int64_t e = 8192 * i + first8<SPLIT>(threadIdx.x, 0, 1024);
            float y[8], v[8], w[8], d[8];
            load8<YT, SPLIT>(dy, e, a.K, y);
            load8<HT, SPLIT>(h, e, a.K, v);
            load8<kF32, SPLIT>(a.w, e, a.K, w);
            if (a.dr) load8<DT, SPLIT>(dr, e, a.K, d);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = v[j] * rstd;
                const float g = rstd * (y[j] * w[j] - n * mean);
                d[j] = a.dr ? g + d[j] : g;
                if (a.partial && e + at8<SPLIT>(j) < a.K) {
                    float *p = a.partial + static_cast<int64_t>(blockIdx.x) * a.K + e + at8<SPLIT>(j);
                    *p = first ? y[j] * n : *p + y[j] * n;
                }
            }
            store8<DT, SPLIT>(dh, e, a.K, d);
        }
    }
}

// dw[k] = sum over the blocks' shares: 32 columns per block, each of its 32
// warps adds every 32nd share, then warp w adds the 32 sums of column w: a fixed
// order, and all of a warp's loads (at most ten; five of them for the 148 shares
// of a device with 148 SMs) are in flight together.
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float *__restrict__ partial, float *dw, int rows,
                                                          int64_t K) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    wait_for_stream();
    float v[10];
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const int r = warp + 32 * i;
        v[i] = col < K && r < rows ? __ldcg(&partial[r * K + col]) : 0.0f;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 10; ++i) s += v[i];
    part[warp][lane] = s;
    __syncthreads();
    // warp w sums column w over the 32 warps
    s = warp_sum(part[lane][warp]);
    const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + warp;
    if (lane == 0 && out < K) dw[out] = s;
}

}  // namespace b200
