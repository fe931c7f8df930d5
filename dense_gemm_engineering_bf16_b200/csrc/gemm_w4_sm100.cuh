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
// bf16 (over 64 too), so the products are exact and the only roundings are
// those of the fp32 sums and of the output.
//
// Codes to bf16 (w4_codes): one AND and one fused multiply-add per pair.  The
// AND picks nibbles i and i + 4 of a 32-bit word of eight codes, so an MMA's K
// order is 0 4 1 5 2 6 3 7 within each eight; the activations are put in that
// order when they are staged in shared memory.  The weights come out divided by
// 64, which the result makes good, exactly.
//
// A block takes 16 weight rows per warp and a share of K (its rank in a
// cluster).  Every warp streams its own rows through a ring of shared-memory
// stages of 256 K with 16-byte cp.async copies (one 128-byte line per row and
// stage); the activations are shared by the block and staged one stage ahead
// through registers.  The cluster's partial sums meet in distributed shared
// memory and are added in a fixed order: no workspace, and the same result
// every time.
//
// What bounds it: the steps from codes to sums, as far as the copies do not hide
// them.  At 1 x 8192 x 8192 the copies alone take 8.1 us
// (5.3 is the bytes' floor, the rest start and end), with the arithmetic 12.8
// (13.3 with weights from memory rather than L2); at 16 rows 17.0 (17.2).  Per 16
// x 32 weights of 16 rows a warp issues 53 instructions (counted by ncu, groups
// of 128, zeros): 19 in the integer and bit pipe, ten of which unpack codes and
// the rest address, select and permute; 18 multiply-adds; 8 loads and stores; 4
// MMAs.  No pipe is near its rate (tensor 25 %, bits about as much): what is left is
// latency, with 16 warps per SM and a block-wide barrier per stage.  Each
// further 8 rows of a batch cost 2 to 6 us at this size: 25 us at 32, 42.5 at 64 with
// groups of 128, where a bf16 copy of the weights through gemm_bf16 takes 33.
//
// Registers: at 9 to 32 rows the bound of 128 (two blocks per SM) spills up to 48
// bytes, at 9 to 16 rows with groups of 64 only, at 17 to 32 rows with groups of 32,
// 64 and 128; from 33 rows on (255) groups of 32 spill 40 to 84 bytes and groups of
// 64, from 49 rows on, 100.  Groups of 256 and more spill nowhere.  16 x 8192 x 8192
// with groups of 64 takes 19.8 us, of 32 19.3, of 128 17.0; 64 x 8192 x 8192 53.3,
// 56.4 and 42.5.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "rows.cuh"

namespace b200 {

constexpr int kW4K = 256;                    // K per stage
constexpr int kW4Pitch = kW4K / 2 + 16;      // staged row of codes: 144 bytes, conflict-free 32-bit reads
constexpr int kW4StageRow = kW4Pitch + 16 + 8;   // + its scales (16 bytes) and zeros (8 bytes)
constexpr int kW4XPitch = 2 * kW4K + 64;     // staged activation row: conflict-free 16-byte reads

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
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Codes i and i + 4 of a word of eight (I = 0: i = 0, I = 1: i = 1; codes 2, 3,
// 6 and 7 from the word shifted right by 8) as bf16 (q - z) / 64, with `minus`
// the pair -z / 64.  The AND leaves q 16^I in each half, as a bf16 the
// subnormal q 16^I 2^-133 (bf16 patterns below 0x0100 grow linearly through the
// subnormals and the first binade), and one fused multiply-add by 2^127 or
// 2^123 makes q / 64 - z / 64 of it, exactly.  Five bit operations per word;
// without the subnormals it takes seven (16 x 8192 x 8192: 18.5 against 19.0 us).
template <int I>
__device__ __forceinline__ uint32_t w4_codes(uint32_t word, uint32_t minus) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
        : "=r"(d)
        : "r"(word & (I ? 0x00F000F0u : 0x000F000Fu)), "r"(I ? 0x7D007D00u : 0x7F007F00u), "r"(minus));
    return d;
}

// -z / 64 of the byte z = zeros[i], as a bf16 pair.
__device__ __forceinline__ uint32_t w4_minus(uint32_t zeros, int i) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"       // z as a subnormal times -2^127, minus 0
        : "=r"(d)
        : "r"(__byte_perm(zeros, 0u, 0x4040u | 0x101u * i)), "r"(0xFF00FF00u), "r"(0x80008000u));
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
    uint32_t stages;         // ceil(K / kW4K)
    int split_shift;         // log2 of the cluster's size
};

// NT: activation rows in eights; WARPS per block; S: ring stages.
template <int NT_, int WARPS_, int S_>
struct W4Cfg {
    static constexpr int NT = NT_, WARPS = WARPS_, S = S_;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int WROWS = 16;                       // weight rows per warp
    static constexpr int ROWS = WROWS * WARPS;             // and per block
    static constexpr int SLOT_BYTES = WROWS * kW4StageRow;
    static constexpr int RING_BYTES = S * SLOT_BYTES;      // per warp
    static constexpr int X_BYTES = 8 * NT * kW4XPitch;     // activations of one stage, staged twice
    static constexpr int X_ROWS = (8 * NT + WARPS - 1) / WARPS;    // activation rows that a warp stages
    static constexpr int SMEM_BYTES = WARPS * RING_BYTES + 2 * X_BYTES;
    static constexpr int RED_PITCH = ROWS + 4;             // partial sums [token][row], in the rings' place
    static constexpr int PER_SM = SMEM_BYTES <= 112 * 1024 ? 2 : 1;    // blocks that an SM holds
    static_assert(8 * NT * RED_PITCH * 4 <= SMEM_BYTES, "partial sums fit");
};

// Sum over the cluster's SPLIT blocks of the float at one shared address.
template <int SPLIT>
__device__ __forceinline__ float w4_gather(uint32_t at) {
    float f[SPLIT], v = 0.0f;
#pragma unroll
    for (uint32_t p = 0; p < SPLIT; ++p)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f[p]) : "r"(map_to_cta(at, p)));
#pragma unroll
    for (int p = 0; p < SPLIT; ++p) v += f[p];
    return v;
}

// The two bf16 of a pair as fp32.
__device__ __forceinline__ float w4_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float w4_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// U: 32-K steps per scale (G = 32 U; 8 also for larger groups).
template <class Cfg, int U>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::PER_SM) gemm_w4_kernel(W4Args a) {
    constexpr int NT = Cfg::NT, S = Cfg::S, THREADS = Cfg::THREADS, WROWS = Cfg::WROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / 4, t = lane % 4;
    // grid: x = weight tile and K share (the cluster's ranks), y = activation rows
    const uint32_t split = 1u << a.split_shift, rank = blockIdx.x & (split - 1);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x >> a.split_shift) * Cfg::ROWS;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (8 * NT);
    const int tokens = static_cast<int>(min(a.M - m0, static_cast<int64_t>(8 * NT)));
    // at most 2^23 stages of K, split by at most 8
    const uint32_t s_begin = rank * a.stages >> a.split_shift, s_end = (rank + 1) * a.stages >> a.split_shift;

    // this warp's ring; a slot holds codes, then scales, then zeros
    uint8_t *const ring = smem + warp * Cfg::RING_BYTES;
    uint8_t *const x_smem = smem + Cfg::WARPS * Cfg::RING_BYTES;
    if (!a.zeros) {     // zeros of 8 in every slot, once
        for (int i = lane; i < S * WROWS; i += 32)
            *reinterpret_cast<uint2 *>(ring + (i / WROWS) * Cfg::SLOT_BYTES + WROWS * (kW4Pitch + 16) +
                                       8 * (i % WROWS)) = make_uint2(0x08080808u, 0x08080808u);
    }

    // What this lane copies of each stage: 16 bytes (32 codes) of every fourth
    // row, and one row's scales and zeros.  Rows past N repeat the last row
    // (their sums are not stored), so that only the end of K needs a test.
    const int64_t n_warp = n0 + warp * WROWS;
    const uint8_t *codes[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
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
                for (int i = 0; i < 4; ++i)
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
        fill = fill == (S - 1) * Cfg::SLOT_BYTES ? 0 : fill + Cfg::SLOT_BYTES;
        asm volatile("cp.async.commit_group;" ::: "memory");   // one group per stage, empty ones too
    };

    wait_for_stream();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) load_stage(s_begin + i);

    // Activations: warp w stages rows w, w + WARPS, ... of each stage, 32 lanes
    // to a row, in the MMA's K order and zero past K.  Two buffers: the next
    // stage's are loaded while this one is worked on.
    const uint16_t *x_src[Cfg::X_ROWS];
#pragma unroll
    for (int i = 0; i < Cfg::X_ROWS; ++i)
        x_src[i] = a.a + (m0 + min(warp + i * Cfg::WARPS, tokens - 1)) * a.lda + static_cast<int64_t>(s_begin) * kW4K +
                   8 * lane;
    uint4 x_next[Cfg::X_ROWS];
    auto load_x = [&](uint32_t st) {
        const bool in = st < s_end && st * (kW4K / 8) + lane < 4 * k_steps;
#pragma unroll
        for (int i = 0; i < Cfg::X_ROWS; ++i) {
            x_next[i] = make_uint4(0, 0, 0, 0);
            if (in && warp + i * Cfg::WARPS < tokens) x_next[i] = *reinterpret_cast<const uint4 *>(x_src[i]);
            x_src[i] += kW4K;
        }
    };
    auto store_x = [&](uint8_t *buffer) {
#pragma unroll
        for (int i = 0; i < Cfg::X_ROWS; ++i) {
            const uint4 x = x_next[i];
            if (warp + i * Cfg::WARPS < tokens)
                *reinterpret_cast<uint4 *>(buffer + (warp + i * Cfg::WARPS) * kW4XPitch + 16 * lane) =
                    make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                               __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
        }
    };
    // rows of the MMA's columns; columns past the last row repeat it and are not stored
    uint32_t x_row[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) x_row[nt] = min(8 * nt + g, tokens - 1) * kW4XPitch + 16 * t;

    float acc[NT][4] = {};
    uint32_t read = 0;                    // ring slot (byte offset) to read
    uint32_t x_read = 0;                  // and activation buffer
    load_x(s_begin);
    for (uint32_t st = s_begin; st < s_end; ++st) {
        // this buffer was last read two stages ago, before the barrier of the previous one
        store_x(x_smem + x_read);
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        __syncthreads();
        load_x(st + 1);
        load_stage(st + S - 1);           // into the slot read in the previous iteration
        const uint8_t *src = ring + read;
        const uint8_t *xs = x_smem + x_read;
        read = read == (S - 1) * Cfg::SLOT_BYTES ? 0 : read + Cfg::SLOT_BYTES;
        x_read ^= Cfg::X_BYTES;
        // the stage's scales and zeros of this lane's rows: 8 / U groups from g_low on
        const uint32_t g_low = U == 8 ? st >> (a.group_shift - 8) : U == 4 ? 2 * st : 0u;
        constexpr int GROUPS = 8 / U;
        float scale[2][GROUPS];
        uint32_t zero[2][(GROUPS + 3) / 4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 8 * h + g;
            const uint8_t *sc = src + WROWS * kW4Pitch + 16 * row;
            if constexpr (U == 8) {
                scale[h][0] = w4_low(*reinterpret_cast<const uint16_t *>(sc + 2 * (g_low & 1)));
            } else {
#pragma unroll
                for (int i = 0; i < GROUPS / 2; ++i) {
                    const uint32_t w = reinterpret_cast<const uint32_t *>(sc)[i];
                    scale[h][2 * i] = w4_low(w);
                    scale[h][2 * i + 1] = w4_high(w);
                }
            }
            const uint8_t *zr = src + WROWS * (kW4Pitch + 16) + 8 * row;
#pragma unroll
            for (int i = 0; i < (GROUPS + 3) / 4; ++i)
                zero[h][i] = (reinterpret_cast<const uint32_t *>(zr)[i] & 0x0F0F0F0Fu) >> (8 * (g_low & 3));
        }
#pragma unroll
        for (int grp = 0; grp < GROUPS; ++grp) {
            // The two MMAs of a step add to one sum only where other sums stand
            // between them: a dependent MMA waits some 20 cycles.
            constexpr int CHAINS = NT <= 2 ? 2 : 1;
            float part[CHAINS][NT][4];
            uint32_t minus[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) minus[h] = w4_minus(zero[h][grp / 4], grp % 4);
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
                const uint8_t *w = src + g * kW4Pitch + 16 * j + 4 * t;
                const uint32_t lo = *reinterpret_cast<const uint32_t *>(w);
                const uint32_t hi = *reinterpret_cast<const uint32_t *>(w + 8 * kW4Pitch);
                const uint32_t a0[4] = {w4_codes<0>(lo, minus[0]), w4_codes<0>(hi, minus[1]),
                                        w4_codes<1>(lo, minus[0]), w4_codes<1>(hi, minus[1])};
                const uint32_t a1[4] = {w4_codes<0>(lo >> 8, minus[0]), w4_codes<0>(hi >> 8, minus[1]),
                                        w4_codes<1>(lo >> 8, minus[0]), w4_codes<1>(hi >> 8, minus[1])};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float (&p)[4] = part[0][nt];
                    if (u == 0) w4_mma(p, a0, x[nt][0], x[nt][1], 0.0f, 0.0f, 0.0f, 0.0f);
                    else w4_mma(p, a0, x[nt][0], x[nt][1], p[0], p[1], p[2], p[3]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float (&p)[4] = part[CHAINS - 1][nt];
                    if (u == 0 && CHAINS == 2) w4_mma(p, a1, x[nt][2], x[nt][3], 0.0f, 0.0f, 0.0f, 0.0f);
                    else w4_mma(p, a1, x[nt][2], x[nt][3], p[0], p[1], p[2], p[3]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float p = part[0][nt][r];
                    if (CHAINS == 2) p += part[1][nt][r];
                    acc[nt][r] += scale[r / 2][grp] * p;
                }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // partial sums [token][row] over the rings
    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            red[(8 * nt + 2 * t + (r & 1)) * Cfg::RED_PITCH + warp * WROWS + g + 8 * (r / 2)] = acc[nt][r];
    if (split > 1) cluster_sync_all();
    else __syncthreads();
    // Rank r writes its share of the rows, summed in rank order; the shares of
    // an output are read together (one after the other their latencies through
    // the cluster would add up).
    const int rows = Cfg::ROWS >> a.split_shift, row0 = rows * static_cast<int>(rank);     // a power of two
    const int row_shift = 31 - __clz(rows);
    const uint32_t red_addr = smem_addr(red);
    for (int i = tid; i < tokens << row_shift; i += THREADS) {
        const int token = i >> row_shift, row = row0 + (i & (rows - 1));
        const uint32_t at = red_addr + 4 * (token * Cfg::RED_PITCH + row);
        float v;
        if (a.split_shift == 3) v = w4_gather<8>(at);
        else if (a.split_shift == 2) v = w4_gather<4>(at);
        else if (a.split_shift == 1) v = w4_gather<2>(at);
        else v = red[token * Cfg::RED_PITCH + row];
        v *= 64.0f;         // the weights went in over 64
        if (n0 + row < a.N) {
            const int64_t o = (m0 + token) * a.ldc + n0 + row;
            if (a.out == kF32) static_cast<float *>(a.c)[o] = v;
            else static_cast<__nv_bfloat16 *>(a.c)[o] = __float2bfloat16_rn(v);
        }
    }
    if (split > 1) cluster_sync_all();   // no block leaves while another reads its sums
}

}  // namespace b200
