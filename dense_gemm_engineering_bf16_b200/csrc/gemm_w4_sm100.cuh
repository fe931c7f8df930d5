// C = A . dequant(B): bf16 activations, 4-bit weights with group scales.
//
//   c[i][j] = sum_k a[i][k] * s[j][k / G] * (q[j][k] - z[j][k / G])
//
// For the few rows of a decoding batch the weights' bytes are the bound, so
// every SM streams its share of them once and the arithmetic has to keep out
// of the way: codes go to bf16 without conversions, the products run on the
// warp-level tensor instruction mma.sync m16n8k16 with 16 weight rows as its
// M and 8 activation rows as its N, and the scale is applied to the fp32 sum
// of a group, not to each weight.  q - z is an integer in [-15, 15], exact in
// bf16, so the products are exact and the only roundings are those of the
// fp32 sums and of the output.
//
// Codes to bf16: the bits 0x4300 | q are the bf16 number 128 + q (its last
// place is 1 there), so two codes sit ready after one AND-OR, and subtracting
// 128 + z, exact as well, leaves q - z.  The AND-OR picks nibbles i and i + 4 of
// a 32-bit word of eight codes, so an MMA's K order is 0 4 1 5 2 6 3 7 within
// each eight; the activations are put in that order once, when they are
// staged in shared memory.
//
// A block takes 128 weight rows and a share of K (cluster rank r of s), its
// warps 16 * MT rows each.  Every warp streams its own rows through a ring of
// shared-memory stages of 256 K with 16-byte cp.async copies (one 128-byte
// line per row and stage) and synchronises with no other warp for it.  The
// cluster's partial sums meet in distributed shared memory and are added in
// rank order: no workspace, and the same result every time.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "rows.cuh"

namespace b200 {

constexpr int kW4Rows = 128;                 // weight rows per block
constexpr int kW4K = 256;                    // K per stage
constexpr int kW4Pitch = kW4K / 2 + 16;      // staged row of codes: 144 bytes, conflict-free 32-bit reads
constexpr int kW4StageRow = kW4Pitch + 16 + 8;   // + its scales (16 bytes) and zeros (8 bytes)
constexpr int kW4StageBytes = kW4Rows * kW4StageRow;
constexpr int kW4RedPitch = kW4Rows + 4;     // partial sums [token][row]

// Copies of 4, 8 or 16 bytes, the first `bytes` of them read, the rest zero.
template <int SIZE>
__device__ __forceinline__ void w4_copy(uint32_t dst, const void *src, uint32_t bytes) {
    if constexpr (SIZE == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(SIZE), "r"(bytes)
                     : "memory");
}

__device__ __forceinline__ void w4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes (4 * i .. i) and (i + 4) of a word of eight as bf16 q - z.
template <int I>
__device__ __forceinline__ uint32_t w4_codes(uint32_t word, __nv_bfloat162 zero) {
    const uint32_t t = ((word >> (4 * I)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&t), zero);
    return *reinterpret_cast<const uint32_t *>(&d);
}

struct W4Args {
    const uint16_t *a;
    const uint8_t *b;
    const uint16_t *scales;
    const uint8_t *zeros;    // null: 8 everywhere
    void *c;
    int64_t M, N, K, lda, ldb, lds, ldc;
    int64_t groups;          // ceil(K / G)
    int group_shift;         // log2 G
    int out;                 // kF32 or kBF16
    int token_blocks;        // ceil(M / (8 * NT))
    int x_stages;            // stages of K whose activations are staged at a time
    int x_pitch;             // bytes per staged activation row
};

// NT: activation rows in eights; MT: weight rows per warp in sixteens; U: 32-K
// steps per scale (G = 32 U; 8 also for larger groups); S: ring stages.
template <int NT, int MT, int U, int S>
__global__ void __launch_bounds__(32 * (kW4Rows / (16 * MT))) gemm_w4_kernel(W4Args a) {
    constexpr int WARPS = kW4Rows / (16 * MT);
    constexpr int THREADS = 32 * WARPS;
    constexpr int WROWS = 16 * MT;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / 4, t = lane % 4;
    const uint32_t split = cluster_num_ctas(), rank = cluster_cta_rank();
    const int64_t unit = blockIdx.x / split;
    const int64_t n0 = unit / a.token_blocks * kW4Rows;
    const int64_t m0 = unit % a.token_blocks * (8 * NT);
    const int tokens = static_cast<int>(min(a.M - m0, static_cast<int64_t>(8 * NT)));
    const int64_t stages = (a.K + kW4K - 1) / kW4K;
    const int64_t s_begin = rank * stages / split, s_end = (rank + 1) * stages / split;

    uint8_t *const x_smem = smem + S * kW4StageBytes;
    // this warp's part of stage slot b: codes, then scales, then zeros
    auto slot = [&](int b) { return smem + b * kW4StageBytes + warp * WROWS * kW4StageRow; };

    auto load_stage = [&](int64_t st) {
        if (st < s_end) {
            uint8_t *dst = slot(static_cast<int>((st - s_begin) % S));
            const int64_t k0 = st * kW4K;
#pragma unroll
            for (int i = 0; i < 4 * MT; ++i) {
                const int row = (lane >> 3) + 4 * i;
                const int64_t n = n0 + warp * WROWS + row, k = k0 + 32 * (lane & 7);
                const bool in = n < a.N && k < a.K;     // K is a multiple of 32: whole copies
                w4_copy<16>(smem_addr(dst + row * kW4Pitch + 16 * (lane & 7)), in ? a.b + n * a.ldb + k / 2 : a.b,
                            in ? 16u : 0u);
            }
            // per row the stage's scales, in one copy from a multiple of its size
            const int64_t g0 = k0 >> a.group_shift;
            {
                constexpr int BYTES = U == 1 ? 16 : U == 2 ? 8 : 4;
                const int64_t first = g0 & ~static_cast<int64_t>(BYTES / 2 - 1);
                const int64_t left = 2 * (a.groups - first);
                const int64_t n = n0 + warp * WROWS + lane;
                if (lane < WROWS)
                    w4_copy<BYTES>(smem_addr(dst + WROWS * kW4Pitch + 16 * lane),
                                   n < a.N ? a.scales + n * a.lds + first : a.scales,
                                   n < a.N ? static_cast<uint32_t>(left < BYTES ? left : BYTES) : 0u);
            }
            if (a.zeros) {
                constexpr int BYTES = U == 1 ? 8 : 4;
                const int64_t first = g0 & ~static_cast<int64_t>(BYTES - 1);
                const int64_t left = a.groups - first;
                const int64_t n = n0 + warp * WROWS + lane;
                if (lane < WROWS)
                    w4_copy<BYTES>(smem_addr(dst + WROWS * (kW4Pitch + 16) + 8 * lane),
                                   n < a.N ? a.zeros + n * a.lds + first : a.zeros,
                                   n < a.N ? static_cast<uint32_t>(left < BYTES ? left : BYTES) : 0u);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");   // one group per stage, empty ones too
    };

#pragma unroll
    for (int i = 0; i < S - 1; ++i) load_stage(s_begin + i);

    float acc[MT][NT][4] = {};
    int x_left = 0;                 // stages whose activations are still staged
    int64_t x_first = s_begin;
    for (int64_t st = s_begin; st < s_end; ++st) {
        if (x_left == 0) {
            // activations of the next stages, in the MMA's K order, zero past K
            if (st != s_begin) __syncthreads();
            x_first = st;
            x_left = static_cast<int>(min(static_cast<int64_t>(a.x_stages), s_end - st));
            const int vecs = x_left * (kW4K / 8);
            for (int i = tid; i < tokens * vecs; i += THREADS) {
                const int row = i / vecs, v = i % vecs;
                const int64_t k = st * kW4K + 8 * v;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (k < a.K) x = *reinterpret_cast<const uint4 *>(a.a + (m0 + row) * a.lda + k);
                *reinterpret_cast<uint4 *>(x_smem + row * a.x_pitch + 16 * v) =
                    make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                               __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
            }
            __syncthreads();
        }
        --x_left;
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();
        load_stage(st + S - 1);     // into the slot read in the previous iteration
        const uint8_t *src = slot(static_cast<int>((st - s_begin) % S));
        const int64_t g0 = (st * kW4K) >> a.group_shift;
        const uint8_t *sc = src + WROWS * kW4Pitch + (U >= 4 ? 2 * (g0 & 1) : 0);
        const uint8_t *zr = src + WROWS * (kW4Pitch + 16) + (U >= 4 ? (g0 & 3) : 0);
        const uint8_t *xs = x_smem + (st - x_first) * (2 * kW4K) + 16 * t;
#pragma unroll
        for (int grp = 0; grp < 8 / U; ++grp) {
            float part[MT][NT][4] = {};
            __nv_bfloat162 zero[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t z = a.zeros ? zr[8 * (16 * mt + 8 * h + g) + grp] & 15u : 8u;
                    const uint32_t zz = (0x4300u | z) * 0x10001u;
                    zero[mt][h] = *reinterpret_cast<const __nv_bfloat162 *>(&zz);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = grp * U + u;
                uint32_t x[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int row = min(8 * nt + g, tokens - 1);    // columns past the last row are not stored
                    const uint4 v = *reinterpret_cast<const uint4 *>(xs + row * a.x_pitch + 64 * j);
                    x[nt][0] = v.x;
                    x[nt][1] = v.y;
                    x[nt][2] = v.z;
                    x[nt][3] = v.w;
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint8_t *w = src + (16 * mt + g) * kW4Pitch + 16 * j + 4 * t;
                    const uint32_t lo = *reinterpret_cast<const uint32_t *>(w);
                    const uint32_t hi = *reinterpret_cast<const uint32_t *>(w + 8 * kW4Pitch);
                    const uint32_t a0[4] = {w4_codes<0>(lo, zero[mt][0]), w4_codes<0>(hi, zero[mt][1]),
                                            w4_codes<1>(lo, zero[mt][0]), w4_codes<1>(hi, zero[mt][1])};
                    const uint32_t a1[4] = {w4_codes<2>(lo, zero[mt][0]), w4_codes<2>(hi, zero[mt][1]),
                                            w4_codes<3>(lo, zero[mt][0]), w4_codes<3>(hi, zero[mt][1])};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        w4_mma(part[mt][nt], a0, x[nt][0], x[nt][1]);
                        w4_mma(part[mt][nt], a1, x[nt][2], x[nt][3]);
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float s[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    s[h] = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(
                                               sc + 16 * (16 * mt + 8 * h + g) + 2 * grp))
                                           << 16);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[mt][nt][r] += s[r / 2] * part[mt][nt][r];
            }
        }
        __syncwarp();               // the slot may be overwritten from the next iteration on
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // partial sums [token][row] over the ring
    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                red[(8 * nt + 2 * t + (r & 1)) * kW4RedPitch + warp * WROWS + 16 * mt + g + 8 * (r / 2)] =
                    acc[mt][nt][r];
    if (split > 1) cluster_sync_all();
    else __syncthreads();
    // rank r writes rows [128 r / s, 128 (r + 1) / s), summed in rank order
    const int rows = kW4Rows / static_cast<int>(split), row0 = rows * static_cast<int>(rank);
    for (int i = tid; i < tokens * rows; i += THREADS) {
        const int token = i / rows, row = row0 + i % rows;
        const uint32_t at = smem_addr(red + token * kW4RedPitch + row);
        float v = 0.0f;
        for (uint32_t p = 0; p < split; ++p) {
            float f;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(map_to_cta(at, p)) : "memory");
            v += f;
        }
        if (n0 + row < a.N) {
            const int64_t o = (m0 + token) * a.ldc + n0 + row;
            if (a.out == kF32) static_cast<float *>(a.c)[o] = v;
            else static_cast<__nv_bfloat16 *>(a.c)[o] = __float2bfloat16_rn(v);
        }
    }
    if (split > 1) cluster_sync_all();   // no block leaves while another reads its sums
}

}  // namespace b200
