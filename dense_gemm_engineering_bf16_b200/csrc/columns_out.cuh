// Write-back of products whose accumulator lies the other way round than C: a
// TMEM lane is a column of C, a TMEM column one of its rows.  Four warps, one per
// lane quarter, hold 128 columns of C.
//
// bf16: tcgen05.ld 16x256b gives a thread two neighbouring rows of one column;
// packed, they are a fragment that stmatrix.trans writes to shared memory as
// rows, from where they go out as 16 bytes a lane, whole lines of 128 bytes: about
// 50 instructions for 32 x 32 values.  (Straight from the registers, a column a
// lane, they took 400: with two such warps per scheduler that, not memory, was
// the time, 5.6 us for a 256 x 256 tile, now 3.0, of which 1.7 are the stores.
// One bulk copy per row of 256 bytes is bound by the copies, about 20 cycles
// each; 32-byte stores of a row a lane take 20 % longer.)
//
// fp32: a lane's column straight from its registers, a line per row and warp.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "rows.cuh"

namespace b200 {

// 16 lanes x 32 columns: thread t gets of lane t / 4 (and t / 4 + 8) the columns
// 8 i + 2 (t % 4) and the next in r[4 i], r[4 i + 1] (r[4 i + 2], r[4 i + 3]).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// 32 rows x 32 columns of this warp: `from` its quarter's first row in TMEM.
__device__ __forceinline__ void load_rows(uint32_t from, uint32_t (&lo)[16], uint32_t (&hi)[16]) {
    tmem_ld_16x256b_x4(from, lo);
    tmem_ld_16x256b_x4(from + (16u << 16), hi);
}

// Packed as bf16 once they have arrived: w[8 h + 2 i + p] has lanes 16 h + 8 p + t / 4,
// rows 8 i + 2 (t % 4).
__device__ __forceinline__ void pack_rows(float alpha, const uint32_t (&lo)[16], const uint32_t (&hi)[16],
                                          uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = pack_bf16x2(alpha * __uint_as_float(lo[2 * i]), alpha * __uint_as_float(lo[2 * i + 1]));
        w[8 + i] = pack_bf16x2(alpha * __uint_as_float(hi[2 * i]), alpha * __uint_as_float(hi[2 * i + 1]));
    }
}

// N chunks of 32 rows, `stride` TMEM columns apart, two of them on their way at
// a time (registers).
template <int N>
__device__ __forceinline__ void load_chunks_bf16(uint32_t from, uint32_t stride, float alpha, uint32_t (&w)[N][16]) {
    uint32_t lo[2][16], hi[2][16];
#pragma unroll
    for (int c = 0; c < N; c += 2) {
#pragma unroll
        for (int i = 0; i < 2 && c + i < N; ++i) load_rows(from + (c + i) * stride, lo[i], hi[i]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 2 && c + i < N; ++i) pack_rows(alpha, lo[i], hi[i], w[c + i]);
    }
}

constexpr int kOutHalf = 32 * 128;              // 32 rows x 64 columns of bf16
constexpr int kOutBytes = 2 * 2 * kOutHalf;     // two buffers of 128 columns for each four warps

// Where a warp's bf16 rows go.  The warps of two neighbouring quarters share 64
// columns, a line of 128 bytes per row; they call every member together.
struct ColumnsOut {
    uint32_t buffer;        // the two warps' shared memory: two of kOutHalf bytes
    uint32_t barrier;       // their named barrier
    uint32_t quarter, lane;
    int64_t ld_bytes;
    int cols;               // of C from the four warps' first one on; may be none
    uint32_t turn;

    __device__ __forceinline__ ColumnsOut(uint32_t base, uint32_t part, uint32_t sub, uint32_t lane_, int64_t ld)
        : buffer(base + part * kOutBytes + sub / 2 * 2 * kOutHalf), barrier(1 + 2 * part + sub / 2), quarter(sub),
          lane(lane_), ld_bytes(ld), cols(0), turn(0) {}

    // Whether neither warp failed.
    __device__ __forceinline__ bool agree(bool ok) {
        uint32_t both;
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                     "barrier.red.and.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(both) : "r"(ok ? 1u : 0u), "r"(barrier) : "memory");
        return both != 0;
    }

    // 32 rows from pack_rows, the first `count` of them to C's from `c` on
    // (the four warps' first column).  Rows are 128 bytes in shared memory, their
    // 16-byte pieces swapped by row, so that neither direction has bank
    // conflicts.  The barrier also says that both warps have read the other
    // buffer, which the next rows go to.
    __device__ __forceinline__ void rows(const uint32_t (&w)[16], uint8_t *c, int count) {
        const uint32_t at = buffer + turn * kOutHalf;
        // matrix m of a store: rows of C 8 (m / 2) .., columns 8 (m % 2) .. of 16
        const uint32_t m = lane >> 3, r0 = 8 * (m >> 1) + (lane & 7), piece = 4 * (quarter & 1) + (m & 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                stmatrix_x4_trans(at + (r0 + 8 * i) * 128 + (((piece + 2 * h) ^ (r0 & 7)) << 4), w[8 * h + 2 * i],
                                  w[8 * h + 2 * i + 1], w[8 * h + 2 * i + 2], w[8 * h + 2 * i + 3]);
        asm volatile("bar.sync %0, 64;" ::"r"(barrier) : "memory");
        const int col = 64 * (quarter >> 1) + 8 * (lane & 7), left = cols - col;
        int r = 16 * (quarter & 1) + (lane >> 3);
        uint8_t *p = c + r * ld_bytes + 2 * col;
#pragma unroll
        for (int i = 0; i < 4; ++i, r += 4, p += 4 * ld_bytes) {
            uint32_t v[4];
            ld_shared_v4(at + r * 128 + (((lane & 7) ^ (r & 7)) << 4), v[0], v[1], v[2], v[3]);
            if (r < count && left > 0) {
                if (left >= 8) {
                    *reinterpret_cast<uint4 *>(p) = make_uint4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 7; ++k)
                        if (k < left) reinterpret_cast<uint16_t *>(p)[k] = static_cast<uint16_t>(v[k / 2] >> 16 * (k & 1));
                }
            }
        }
        turn ^= 1u;
    }
};

// W rows of C straight from the registers, a column a lane (`mine`: it is C's):
// the first `rows` of them, C = v + beta * C, rounded once.
template <int W>
__device__ __forceinline__ void store_columns(uint8_t *c, int64_t ld_bytes, int rows, bool mine, bool f32, float beta,
                                              const float *v) {
    if (!mine) return;
    if (f32 && beta == 0.0f) {
#pragma unroll
        for (int j = 0; j < W; ++j, c += ld_bytes)
            if (j < rows) *reinterpret_cast<float *>(c) = v[j];
        return;
    }
#pragma unroll
    for (int j = 0; j < W; ++j, c += ld_bytes) {
        if (j >= rows) break;
        if (f32) {
            float *p = reinterpret_cast<float *>(c);
            *p = fmaf(beta, *p, v[j]);
        } else {
            __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(c);
            *p = __float2bfloat16_rn(beta != 0.0f ? fmaf(beta, __bfloat162float(*p), v[j]) : v[j]);
        }
    }
}

// What sums are multiplied with: ga gb in fp32, except where fp32 would not hold
// that as a normal number (scales are from 2^-100 to 2^100).  Then 2^-100 or
// 2^100 of it come second, so that a sum of zero stays zero and one that brings
// the result back into range is not lost.
struct Factor {
    float first, second;    // second: else 1

    __device__ __forceinline__ Factor(float ga, float gb) : first(ga * gb), second(1.0f) {
        if (fabsf(first) < 0x1p-126f) {
            first = ga * 0x1p100f * gb;
            second = 0x1p-100f;
        } else if (fabsf(first) > 0x1.fffffep127f) {
            first = ga * 0x1p-100f * gb;
            second = 0x1p100f;
        }
    }
    __device__ __forceinline__ float operator()(float sum) const { return sum * first * second; }
};

// Sum over a cluster's members, each of which has the same rows x 128 of C over
// its share of the reduction in TMEM at `acc` (the warp's quarter): `fours` times
// four rows, the first `count` rows are C's.  Member o sums the fours [o share,
// (o + 1) share): the others send theirs to its shared memory (`parts`, 16 bytes
// per four, member and column; `received` counts 128 arrivals from each), and it
// adds all members' in their order and writes them to `c` (the first row of the
// lane's column).  `wait` waits for `received`; false: it failed.
template <class Wait>
__device__ __forceinline__ bool cluster_sum(uint32_t acc, int fours, int members, int me, uint32_t column, uint32_t parts,
                                            uint32_t received, Wait wait, uint8_t *c, int64_t ld_bytes, int count,
                                            bool mine, bool f32, Factor scale) {
    const int share = (fours + members - 1) / members;
    for (int f = 0; f < fours; f += 8) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(acc + 4 * f, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int owner = (f + i) / share;
            if (f + i < fours && owner != me)
                store_cluster_v4(map_to_cta(parts + 16u * ((me * share + (f + i) - owner * share) * 128u + column), owner),
                                 r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        }
    }
    for (int o = 0; o < members; ++o)      // release: the stores come first
        if (o != me) mbar_arrive_cluster(map_to_cta(received, o));
    if (!wait()) return false;
    for (int f = me * share; f < min(fours, (me + 1) * share); ++f) {
        uint32_t own[4];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(own[0]), "=r"(own[1]), "=r"(own[2]), "=r"(own[3]) : "r"(acc + 4 * f));
        tmem_ld_wait();
        float sum[4] = {};
        for (int m = 0; m < members; ++m) {
            uint32_t x[4] = {own[0], own[1], own[2], own[3]};
            if (m != me) ld_shared_v4(parts + 16u * ((m * share + f - me * share) * 128u + column), x[0], x[1], x[2], x[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] += __uint_as_float(x[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = scale(sum[i]);
        store_columns<4>(c + 4 * f * ld_bytes, ld_bytes, count - 4 * f, mine, f32, 0.0f, sum);
    }
    return true;
}

}  // namespace b200
