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
// A block takes 128 or 256 weight rows and a share of K (cluster rank r of s),
// its warps 16 * MT rows each.  Every warp streams its own rows through a ring of
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

constexpr int kW4K = 256;                    // K per stage
constexpr int kW4Pitch = kW4K / 2 + 16;      // staged row of codes: 144 bytes, conflict-free 32-bit reads
constexpr int kW4StageRow = kW4Pitch + 16 + 8;   // + its scales (16 bytes) and zeros (8 bytes)

// Asynchronous copy of 4, 8 or 16 bytes.  (The form with a byte count in a
// register costs several instructions and a branch per copy; here the ends of
// rows are handled by not copying.)
template <int SIZE>
__device__ __forceinline__ void w4_copy(uint32_t dst, const void *src) {
    if constexpr (SIZE == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(SIZE) : "memory");
}

// d = A . B + c; with c = 0 given as constants no register has to be cleared.
__device__ __forceinline__ void w4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                       float c1, float c2, float c3) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Codes i and i + 4 of a word of eight as bf16 q - z, with `minus` the pair
// -(128 + z).  `mask` and `one28` come in registers of their own: as literals
// the AND and the OR would be two instructions, since one takes one literal.
template <int I>
__device__ __forceinline__ uint32_t w4_codes(uint32_t word, uint32_t minus, uint32_t mask, uint32_t one28) {
    uint32_t t, d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(t) : "r"(word >> (4 * I)), "r"(mask), "r"(one28));   // (a & b) | c
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(t), "r"(0x3F803F80u), "r"(minus));
    return d;
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
    int x_shift;             // log2 of the 16-byte vectors per staged activation row
    int x_pitch;             // bytes per staged activation row
};

// NT: activation rows in eights; MT: weight rows per warp in sixteens; WARPS
// per block; S: ring stages.
template <int NT_, int MT_, int WARPS_, int S_>
struct W4Cfg {
    static constexpr int NT = NT_, MT = MT_, WARPS = WARPS_, S = S_;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int WROWS = 16 * MT;                  // weight rows per warp
    static constexpr int ROWS = WROWS * WARPS;             // and per block
    static constexpr int STAGE_BYTES = ROWS * kW4StageRow;
    static constexpr int RING_BYTES = S * STAGE_BYTES;
    static constexpr int RED_PITCH = ROWS + 4;             // partial sums [token][row], over the ring
    static constexpr int X_BYTES = 32 * 1024;              // staged activations, one stage of K at least
    static constexpr int X_STAGE = 8 * NT * 2 * kW4K;
    static constexpr int MAX_SMEM = RING_BYTES + (X_BYTES > X_STAGE ? X_BYTES : X_STAGE) + 8 * NT * 64;
    static_assert(8 * NT * RED_PITCH * 4 <= RING_BYTES, "partial sums fit into the ring");
};

// U: 32-K steps per scale (G = 32 U; 8 also for larger groups).
template <class Cfg, int U>
__global__ void __launch_bounds__(Cfg::THREADS) gemm_w4_kernel(W4Args a) {
    constexpr int NT = Cfg::NT, MT = Cfg::MT, S = Cfg::S, THREADS = Cfg::THREADS, WROWS = Cfg::WROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / 4, t = lane % 4;
    const uint32_t split = cluster_num_ctas(), rank = cluster_cta_rank();
    const int64_t unit = blockIdx.x / split;
    const int64_t n0 = unit / a.token_blocks * Cfg::ROWS;
    const int64_t m0 = unit % a.token_blocks * (8 * NT);
    const int tokens = static_cast<int>(min(a.M - m0, static_cast<int64_t>(8 * NT)));
    const uint32_t stages = static_cast<uint32_t>((a.K + kW4K - 1) / kW4K);
    const uint32_t s_begin = static_cast<uint32_t>(static_cast<uint64_t>(rank) * stages / split);
    const uint32_t s_end = static_cast<uint32_t>(static_cast<uint64_t>(rank + 1) * stages / split);

    // this warp's part of a ring slot: codes, then scales, then zeros
    uint8_t *const ring = smem + warp * WROWS * kW4StageRow;
    uint8_t *const x_smem = smem + Cfg::RING_BYTES;

    // What this lane copies of each stage: 16 bytes (32 codes) of every fourth
    // row, and one row's scales and zeros.  Rows past N repeat the last row
    // (their sums are not stored), so that only the end of K needs a test.
    const int64_t n_warp = n0 + warp * WROWS;
    const uint8_t *codes[4 * MT];
#pragma unroll
    for (int i = 0; i < 4 * MT; ++i)
        codes[i] = a.b + min(n_warp + (lane >> 3) + 4 * i, a.N - 1) * a.ldb + 16 * (lane & 7);
    const uint32_t codes_dst = smem_addr(ring) + (lane >> 3) * kW4Pitch + 16 * (lane & 7);
    const int64_t side_row = min(n_warp + lane % WROWS, a.N - 1) * a.lds;
    const uint16_t *const scale_row = a.scales + side_row;
    const uint8_t *const zero_row = a.zeros ? a.zeros + side_row : nullptr;
    const uint32_t side_dst = smem_addr(ring) + WROWS * kW4Pitch + 16 * (lane % WROWS);
    const uint32_t groups = static_cast<uint32_t>(a.groups), k_steps = static_cast<uint32_t>(a.K / 32);

    uint32_t fill = 0;                    // ring slot (byte offset) of the next copies
    auto load_stage = [&](uint32_t st) {
        if (st < s_end) {
            // K is a multiple of 32, a copy's length.  Codes past K stay what the
            // slot held: any code is finite, and its activations are zero.
            if (st * (kW4K / 32) + (lane & 7) < k_steps) {
#pragma unroll
                for (int i = 0; i < 4 * MT; ++i)
                    w4_copy<16>(codes_dst + fill + 4 * i * kW4Pitch, codes[i] + st * (kW4K / 2));
            }
            // per row the stage's scales and zeros, each in one copy from a
            // multiple of its size; at a row's end one by one, zero past it
            const uint32_t g0 = U == 8 ? st >> (a.group_shift - 8) : st * (8 / U);
            constexpr uint32_t SB = U == 1 ? 16 : U == 2 ? 8 : 4, ZB = U == 1 ? 8 : 4;
            const uint32_t s_first = g0 & ~(SB / 2 - 1), z_first = g0 & ~(ZB - 1);
            if (lane < WROWS) {
                if (s_first + SB / 2 <= groups) {
                    w4_copy<SB>(side_dst + fill, scale_row + s_first);
                } else {
                    for (uint32_t i = 0; i < SB / 2; ++i)
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(side_dst + fill + 2 * i),
                                     "h"(s_first + i < groups ? scale_row[s_first + i] : static_cast<uint16_t>(0))
                                     : "memory");
                }
                const uint32_t zeros_dst = side_dst + fill + 16 * WROWS - 8 * (lane % WROWS);
                if (zero_row) {
                    if (z_first + ZB <= groups) {
                        w4_copy<ZB>(zeros_dst, zero_row + z_first);
                    } else {
                        for (uint32_t i = 0; i < ZB && z_first + i < groups; ++i)
                            asm volatile("st.shared.u8 [%0], %1;" ::"r"(zeros_dst + i),
                                         "h"(static_cast<uint16_t>(zero_row[z_first + i]))
                                         : "memory");
                    }
                }
            }
        }
        fill = fill == (S - 1) * Cfg::STAGE_BYTES ? 0 : fill + Cfg::STAGE_BYTES;
        asm volatile("cp.async.commit_group;" ::: "memory");   // one group per stage, empty ones too
    };

#pragma unroll
    for (int i = 0; i < S - 1; ++i) load_stage(s_begin + i);

    // activation rows of the MMA's columns; columns past the last row repeat it and are not stored
    uint32_t x_row[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) x_row[nt] = min(8 * nt + g, tokens - 1) * a.x_pitch + 16 * t;

    uint32_t mask, one28;                 // kept in registers
    asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x43004300;" : "=r"(one28));
    float acc[MT][NT][4] = {};
    const uint32_t x_stages = 1u << (a.x_shift - 5);    // stages staged at a time
    uint32_t x_at = x_stages;             // next of them
    uint32_t read = 0;                    // ring slot (byte offset) to read
    for (uint32_t st = s_begin; st < s_end; ++st) {
        if (x_at == x_stages) {
            // activations of the next stages, in the MMA's K order, zero past
            // K; several loads in flight per thread
            if (st != s_begin) __syncthreads();
            const int64_t k_end = min(a.K, static_cast<int64_t>(s_end) * kW4K);
            const int total = tokens << a.x_shift;
            for (int i0 = tid; i0 < total; i0 += 8 * THREADS) {
                uint4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int v = i0 + i * THREADS;
                    const int64_t k = static_cast<int64_t>(st) * kW4K + 8 * (v & ((1 << a.x_shift) - 1));
                    x[i] = make_uint4(0, 0, 0, 0);
                    if (v < total && k < k_end)
                        x[i] = *reinterpret_cast<const uint4 *>(a.a + (m0 + (v >> a.x_shift)) * a.lda + k);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int v = i0 + i * THREADS;
                    if (v < total)
                        *reinterpret_cast<uint4 *>(x_smem + (v >> a.x_shift) * a.x_pitch +
                                                   16 * (v & ((1 << a.x_shift) - 1))) =
                            make_uint4(__byte_perm(x[i].x, x[i].z, 0x5410), __byte_perm(x[i].x, x[i].z, 0x7632),
                                       __byte_perm(x[i].y, x[i].w, 0x5410), __byte_perm(x[i].y, x[i].w, 0x7632));
                }
            }
            __syncthreads();
            x_at = 0;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncwarp();
        load_stage(st + S - 1);     // into the slot read in the previous iteration
        const uint8_t *src = ring + read;
        read = read == (S - 1) * Cfg::STAGE_BYTES ? 0 : read + Cfg::STAGE_BYTES;
        const uint32_t g_low = U == 8 ? st >> (a.group_shift - 8) : U == 4 ? 2 * st : 0u;
        const uint8_t *sc = src + WROWS * kW4Pitch + 2 * (g_low & 1);
        const uint8_t *zr = src + WROWS * (kW4Pitch + 16) + (g_low & 3);
        const uint8_t *xs = x_smem + x_at * (2 * kW4K);
        ++x_at;
#pragma unroll
        for (int grp = 0; grp < 8 / U; ++grp) {
            float part[MT][NT][4];
            uint32_t minus[MT][2];      // -(128 + z), twice
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t z = a.zeros ? zr[8 * (16 * mt + 8 * h + g) + grp] & 15u : 8u;
                    minus[mt][h] = (0xC300u | z) * 0x10001u;
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = grp * U + u;
                uint32_t x[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(xs + x_row[nt] + 64 * j);
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
                    uint32_t a0[4], a1[4];
                    a0[0] = w4_codes<0>(lo, minus[mt][0], mask, one28);
                    a0[1] = w4_codes<0>(hi, minus[mt][1], mask, one28);
                    a0[2] = w4_codes<1>(lo, minus[mt][0], mask, one28);
                    a0[3] = w4_codes<1>(hi, minus[mt][1], mask, one28);
                    a1[0] = w4_codes<2>(lo, minus[mt][0], mask, one28);
                    a1[1] = w4_codes<2>(hi, minus[mt][1], mask, one28);
                    a1[2] = w4_codes<3>(lo, minus[mt][0], mask, one28);
                    a1[3] = w4_codes<3>(hi, minus[mt][1], mask, one28);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float (&p)[4] = part[mt][nt];
                        if (u == 0) w4_mma(p, a0, x[nt][0], x[nt][1], 0.0f, 0.0f, 0.0f, 0.0f);
                        else w4_mma(p, a0, x[nt][0], x[nt][1], p[0], p[1], p[2], p[3]);
                        w4_mma(p, a1, x[nt][2], x[nt][3], p[0], p[1], p[2], p[3]);
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
                red[(8 * nt + 2 * t + (r & 1)) * Cfg::RED_PITCH + warp * WROWS + 16 * mt + g + 8 * (r / 2)] =
                    acc[mt][nt][r];
    if (split > 1) cluster_sync_all();
    else __syncthreads();
    // rank r writes its share of the rows, summed in rank order
    const int rows = Cfg::ROWS / static_cast<int>(split), row0 = rows * static_cast<int>(rank);
    for (int i = tid; i < tokens * rows; i += THREADS) {
        const int token = i / rows, row = row0 + i % rows;
        const uint32_t at = smem_addr(red + token * Cfg::RED_PITCH + row);
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
