// Product of 4-bit floating-point operands on the block-scaled tensor cores:
//
//   C[i][j] = ga gb sum_k (a_ik sfa) (b_jk sfb)
//
// E2M1 A (M x K) and B (N x K), one scale per 32 (E8M0) or 16 (E4M3) K elements
// of a row, fp32 accumulation in TMEM.  B's rows run along the MMA's M (128 a
// CTA, TMEM lanes), A's rows along its N, which is chosen per call in steps of
// 16: one token costs an MMA of N = 16, and the same kernel serves a prompt.
//
// Warps of a CTA:
//   0      TMA producer: B, A (rows of 128 bytes = 256 K, 128-byte swizzle) and
//          the scale tiles of both
//   1      MMA issuer (of the pair's leader), owner of TMEM: four MMAs of K = 64
//          a stage
//   2      scale copier: a stage's scale tiles into one of four to eight TMEM
//          slots, ahead of the MMAs and ordered with them by barriers only
//   3 on   epilogue (columns_out.cuh)
//
// Scales in TMEM: a tile of 128 rows x 4 scales becomes four columns (column
// r / 32, lane r % 32 of every quarter, four bytes).  E4M3: a tile is one
// MMA's; E8M0: two MMAs', the second one takes bytes 2 and 3.
//
// SPLIT: a cluster of 2, 4 or 8 CTAs owns a tile, each over a share of K, and
// their partials meet in distributed shared memory (cluster_sum).
//
// What bounds it: shared memory for pairs (per stage and SM the MMAs read 32 KB,
// TMA writes 38 and the scale copies read 6, 600 cycles at 128 bytes each against
// the MMAs' 512; 707 measured, 590 without the loads, 535 without the MMAs) and
// the power limit: 8192^3 207 to 235 us (5.3 to 4.7 PFLOP/s, tensor pipe 73 %
// busy), 4096 x 8192 x 4096 MX 57 us.  Single CTAs: the MMA of 128 x 128 x 64, 122
// cycles instead of the 64 that its size would take: 512 x 4096 x 4096 8.8 us.
// Few rows: memory and the start and end (3.6 us without any work): one row of
// 8192 x 8192, 37.8 MB, 11.4 us; 64 rows 14.3.
// Fewer scale slots cost time (two: 20 %); beyond five nothing changes, and pairs
// take what TMEM has left, five (NV) or eight (MX).
#pragma once
#include <cstdint>

#include "columns_out.cuh"
#include "fp4_quantize_sm100.cuh"
#include "gemm_bf16_sm100.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace b200 {

template <bool NV_, int CG_, int BQ_, int STAGES_, bool SPLIT_ = false>
struct GemmFp4Cfg {
    static constexpr bool NV = NV_, SPLIT = SPLIT_;
    static constexpr int CG = CG_, BQ = BQ_, STAGES = STAGES_;
    static constexpr int BP_CTA = 128, BP = 128 * CG;    // rows of B
    static constexpr int Q_CTA = BQ / CG;                // rows of A this CTA loads at most
    static constexpr int QBOX = BQ >= 128 ? 32 : 16;     // rows of A per TMA box
    static constexpr int BK = 256, ROW_BYTES = BK / 2;
    static constexpr int MMAS = BK / 64;
    static constexpr int N_STEP = 16 * CG;
    static constexpr int CHUNKS = BK / (4 * kFp4Block<NV>);   // scale tiles along K of a stage
    static constexpr int Q_BLOCKS = BQ > 128 ? BQ / 128 : 1;  // scale tiles of 128 rows of A
    static constexpr int P_BYTES = BP_CTA * ROW_BYTES;
    static constexpr int Q_BYTES = Q_CTA * ROW_BYTES;
    static constexpr int SF_BYTES = CHUNKS * kScaleTile;      // of 128 rows
    static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES + (1 + Q_BLOCKS) * SF_BYTES;
    static constexpr int SF_SLOTS = BQ <= 128 ? 4 : NV ? 5 : 8, SLOT_COLS = 4 * CHUNKS * (1 + Q_BLOCKS);
    static constexpr int ACC_BUFS = BQ > 128 ? 1 : 2;
    static constexpr int SF_COL0 = ACC_BUFS * BQ;
    static constexpr int TMEM_COLS = pow2_at_least(SF_COL0 + SF_SLOTS * SLOT_COLS, 32);
    static constexpr int EPI_WARPS = BQ >= 128 ? 8 : 4;
    static constexpr int EPI0 = 3;
    static constexpr int THREADS = 32 * (EPI0 + EPI_WARPS);
    // full[S], empty[S], tmem_full[2], tmem_empty[2], sf_full[slots], sf_empty[slots], received
    static constexpr int NUM_BARS = 2 * STAGES + 4 + 2 * SF_SLOTS + 1;
    static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
    static constexpr int OUT_OFF = BAR_OFF + (NUM_BARS * 8 + 8 + 127) / 128 * 128;    // + TMEM address, abort flag
    static constexpr int PART_OFF = OUT_OFF + EPI_WARPS / 4 * kOutBytes;              // other members' partials
    static constexpr int SMEM_BYTES = 1024 + PART_OFF + (SPLIT ? BQ * 128 * 4 : 0);
    static_assert(TMEM_COLS <= 512 && STAGE_BYTES % 1024 == 0 && SMEM_BYTES <= 232448, "it fits");
    static_assert(!SPLIT || (CG == 1 && EPI_WARPS == 4), "split: one-CTA tiles");
    static constexpr bool ONE_TILE_M = BQ == 64;            // at most BQ rows of A: one tile along M
    static_assert(ONE_TILE_M || BQ % 128 == 0, "a tile's scales start at a tile of scales");
};

struct GemmFp4Args {
    const float *ga, *gb;       // NV; null: 1
    void *c;
    int64_t ldc;
    int M, N, K;
    int tiles_k;                // scale tiles along K
    bool f32;
    DeviceStatus *status;
    uint64_t timeout_ns;
};

// The epilogue of scales whose product needs a second factor.  Apart from the
// ordinary one, which a branch or that factor slowed down by 1 to 1.5 %.
template <class Cfg>
__device__ __noinline__ void fp4_far_tiles(GemmFp4Args a, Factor scale, uint32_t tmem_base, uint32_t tfull, uint32_t tempty,
                                           volatile uint32_t *abort_flag, uint32_t abort_slot, int first, int step,
                                           uint32_t rank) {
    constexpr int FOURS = Cfg::EPI_WARPS / 4;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = warp & 3u;
    const int part = static_cast<int>(warp - Cfg::EPI0) / 4;
    const int tiles_p = parts_of(a.N, Cfg::BP), tiles_q = parts_of(a.M, Cfg::BQ);
    const int64_t esize = a.f32 ? 4 : 2, ld_bytes = a.ldc * esize;
    uint32_t done = 0;
    for (int tile = first; tile < tiles_p * tiles_q; tile += step, ++done) {
        int tq, tp;
        raster_tile(tile, tiles_q, tiles_p, 8, tq, tp);
        const uint32_t buf = done % Cfg::ACC_BUFS;
        if (!mbar_wait_warp(tfull + 8u * buf, (done / Cfg::ACC_BUFS) & 1u, abort_flag, 3 * a.timeout_ns)) {
            if (lane == 0) record_timeout(a.status, abort_flag, abort_slot, Cfg::CG, kRoleEpilogue * 16 + kBarTmemFull);
            break;
        }
        tc_fence_after_sync();
        const int64_t col = int64_t(tp) * Cfg::BP + rank * Cfg::BP_CTA + sub * 32u + lane;
        uint8_t *out = static_cast<uint8_t *>(a.c) + (static_cast<int64_t>(tq) * Cfg::BQ * a.ldc + col) * esize;
#pragma unroll 1
        for (int j = 32 * part; j < Cfg::BQ; j += 32 * FOURS) {
            uint32_t r[32];
            float v[32];
            tmem_ld_32x32b_x32(tmem_base + ((sub * 32u) << 16) + buf * Cfg::BQ + j, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = scale(__uint_as_float(r[i]));
            store_columns<32>(out + j * ld_bytes, ld_bytes, min(Cfg::BQ, a.M - tq * Cfg::BQ) - j, col < a.N, a.f32, 0.0f, v);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
            if (Cfg::CG == 1) mbar_arrive_local(tempty + 8u * buf);
            else mbar_arrive_cluster(map_to_cta(tempty + 8u * buf, 0));
        }
    }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                const __grid_constant__ CUtensorMap tmSP, const __grid_constant__ CUtensorMap tmSQ, GemmFp4Args a) {
    constexpr int CG = Cfg::CG, STAGES = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t base = smem_addr(smem);
    const uint32_t warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const uint32_t rank = CG == 2 ? cluster_cta_rank() : 0u;
    const uint32_t members = Cfg::SPLIT ? cluster_num_ctas() : 1u, me = Cfg::SPLIT ? cluster_cta_rank() : 0u;
    const int cluster = CG * static_cast<int>(members);

    const uint32_t bar0 = base + Cfg::BAR_OFF;
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
    auto sf_full = [&](uint32_t i) { return bar0 + 8u * (2 * STAGES + 4 + i); };
    auto sf_empty = [&](uint32_t i) { return bar0 + 8u * (2 * STAGES + 4 + Cfg::SF_SLOTS + i); };
    const uint32_t received_bar = bar0 + 8u * (2 * STAGES + 4 + 2 * Cfg::SF_SLOTS);
    const uint32_t tmem_slot = bar0 + 8u * Cfg::NUM_BARS, abort_slot = tmem_slot + 4u;
    volatile uint32_t *tmem_slot_ptr = reinterpret_cast<volatile uint32_t *>(smem + Cfg::BAR_OFF + 8 * Cfg::NUM_BARS);
    volatile uint32_t *abort_flag = tmem_slot_ptr + 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), Cfg::EPI_WARPS * CG);
        }
        for (int i = 0; i < Cfg::SF_SLOTS; ++i) {
            mbar_init(sf_full(i), 1);
            mbar_init(sf_empty(i), 1);
        }
        if (Cfg::SPLIT) mbar_init(received_bar, 128 * (members > 1 ? members - 1 : 1));
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc<CG>(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish<CG>();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (cluster > 1) cluster_sync_all();
    tc_fence_after_sync();
    wait_for_stream();
    const uint32_t tmem_base = static_cast<uint32_t>(uniform(static_cast<int>(*tmem_slot_ptr)));

    const int tiles_p = parts_of(a.N, Cfg::BP), tiles_q = parts_of(a.M, Cfg::BQ);
    const int num_tiles = tiles_p * tiles_q;
    const int blocks = parts_of(a.K, Cfg::BK);
    const int kb0 = static_cast<int>(static_cast<int64_t>(blocks) * me / members);
    const int kb1 = static_cast<int>(static_cast<int64_t>(blocks) * (me + 1) / members);
    const int first = static_cast<int>(blockIdx.x) / cluster, step = static_cast<int>(gridDim.x) / cluster;
    auto mma_n = [&](int tq) {
        const int rows = min(Cfg::BQ, a.M - tq * Cfg::BQ);
        return parts_of(rows, Cfg::N_STEP) * Cfg::N_STEP;
    };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer --
        const bool issue = elect_one();
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        for (int tile = first; ok && tile < num_tiles; tile += step) {
            int tq, tp;
            raster_tile(tile, tiles_q, tiles_p, 8, tq, tp);
            const int p = tp * Cfg::BP + static_cast<int>(rank) * Cfg::BP_CTA;
            const int q_cta = mma_n(tq) / CG, q = tq * Cfg::BQ + static_cast<int>(rank) * q_cta;
            const int boxes = (q_cta + Cfg::QBOX - 1) / Cfg::QBOX;
            const uint32_t bytes = Cfg::P_BYTES + boxes * Cfg::QBOX * Cfg::ROW_BYTES + (1 + Cfg::Q_BLOCKS) * Cfg::SF_BYTES;
            const int sp = p / 128 * a.tiles_k, sq = tq * Cfg::BQ / 128 * a.tiles_k;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_warp(empty_bar(stage), phase ^ 1u, abort_flag, 2 * a.timeout_ns)) {
                    if (issue) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleProducer * 16 + kBarEmpty);
                    ok = false;
                    break;
                }
                const uint32_t p_dst = base + stage * Cfg::STAGE_BYTES, q_dst = p_dst + Cfg::P_BYTES;
                const uint32_t s_dst = q_dst + Cfg::Q_BYTES;
                if (issue) {
                    // bytes are counted by the pair's leader
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), CG * bytes);
                    const uint32_t bar = CG == 2 ? map_to_cta(full_bar(stage), 0) : full_bar(stage);
                    auto load = [&](uint32_t dst, const CUtensorMap *m, int x, int y) {
                        if constexpr (CG == 1) tma_load_2d(dst, m, bar, x, y);
                        else tma_load_2d_pair(dst, m, bar, x, y);
                    };
                    load(p_dst, &tmP, kb * Cfg::ROW_BYTES, p);
                    for (int b = 0; b < boxes; ++b)
                        load(q_dst + Cfg::QBOX * Cfg::ROW_BYTES * b, &tmQ, kb * Cfg::ROW_BYTES, q + Cfg::QBOX * b);
                    load(s_dst, &tmSP, 0, sp + kb * Cfg::CHUNKS);
#pragma unroll
                    for (int b = 0; b < Cfg::Q_BLOCKS; ++b)
                        load(s_dst + Cfg::SF_BYTES * (1 + b), &tmSQ, 0, sq + b * a.tiles_k + kb * Cfg::CHUNKS);
                }
                __syncwarp();
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
        }
        // the MMAs' last releases must land before this CTA exits
        for (int i = 0; ok && i < STAGES; ++i) {
            if (!mbar_wait_warp(empty_bar(stage), phase ^ 1u, abort_flag, 2 * a.timeout_ns)) {
                if (issue) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleProducer * 16 + kBarTail);
                ok = false;
            }
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
    } else if (warp == 1) {
        // ------------------------------------------ MMA issuer (pair leader) --
        if (rank == 0) {
            const uint64_t p_desc0 = sw128_kmajor_desc(base), q_desc0 = sw128_kmajor_desc(base + Cfg::P_BYTES);
            const bool issue = elect_one();
            uint32_t stage = 0, phase = 0, n = 0, done = 0;
            bool ok = true;
            for (int tile = first; ok && tile < num_tiles; tile += step, ++done) {
                int tq, tp;
                raster_tile(tile, tiles_q, tiles_p, 8, tq, tp);
                const uint32_t width = static_cast<uint32_t>(mma_n(tq));
                const uint32_t buf = done % Cfg::ACC_BUFS;
                if (!mbar_wait_warp(tempty_bar(buf), ((done / Cfg::ACC_BUFS) & 1u) ^ 1u, abort_flag, 3 * a.timeout_ns)) {
                    if (issue) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleMma * 16 + kBarTmemEmpty);
                    break;
                }
                const uint32_t acc = tmem_base + buf * Cfg::BQ;
                for (int kb = kb0; kb < kb1; ++kb) {
                    const uint32_t slot = n % Cfg::SF_SLOTS;
                    // the copier waited for the stage's bytes before it copied them
                    if (!mbar_wait_warp(full_bar(stage), phase, abort_flag, a.timeout_ns) ||
                        !mbar_wait_warp(sf_full(slot), (n / Cfg::SF_SLOTS) & 1u, abort_flag, a.timeout_ns)) {
                        if (issue) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleMma * 16 + kBarSfFull);
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    if (issue) {
                        const uint64_t p_desc = p_desc0 + (stage * Cfg::STAGE_BYTES >> 4);
                        const uint64_t q_desc = q_desc0 + (stage * Cfg::STAGE_BYTES >> 4);
                        const uint32_t sp = tmem_base + Cfg::SF_COL0 + slot * Cfg::SLOT_COLS;
                        const uint32_t sq = sp + 4 * Cfg::CHUNKS;
                        const int left = a.K - kb * Cfg::BK;
#pragma unroll
                        for (int j = 0; j < Cfg::MMAS; ++j) {
                            if (64 * j >= left) break;      // the scales there are not this row's
                            const uint32_t chunk = Cfg::NV ? j : j / 2, sf_id = Cfg::NV ? 0 : 2 * (j & 1);
                            mma_fp4_ss<CG, Cfg::NV>(acc, p_desc + 2 * j, q_desc + 2 * j,
                                                    idesc_fp4(Cfg::NV, Cfg::BP, width, sf_id), sp + 4 * chunk,
                                                    sq + 4 * Cfg::Q_BLOCKS * chunk, (kb - kb0) | j ? 1u : 0u);
                        }
                        mma_commit<CG>(empty_bar(stage), 0x3);
                        mma_commit<CG>(sf_empty(slot), 0x1);
                        if (kb + 1 == kb1) mma_commit<CG>(tfull_bar(buf), 0x3);
                    }
                    __syncwarp();
                    ++n;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
        }
    } else if (warp == 2) {
        // ---------------------------------- scale copier (pair leader) --
        if (rank == 0) {
            const bool issue = elect_one();
            uint32_t stage = 0, phase = 0, n = 0;
            bool ok = true;
            for (int tile = first; ok && tile < num_tiles; tile += step) {
                for (int kb = kb0; kb < kb1; ++kb, ++n) {
                    const uint32_t slot = n % Cfg::SF_SLOTS;
                    if (!mbar_wait_warp(sf_empty(slot), ((n / Cfg::SF_SLOTS) & 1u) ^ 1u, abort_flag, 2 * a.timeout_ns) ||
                        !mbar_wait_warp(full_bar(stage), phase, abort_flag, 2 * a.timeout_ns)) {
                        if (issue) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleSfCopy * 16 + kBarSfEmpty);
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    if (issue) {
                        const uint64_t src = rows16_desc(base + Cfg::P_BYTES + Cfg::Q_BYTES) + (stage * Cfg::STAGE_BYTES >> 4);
                        const uint32_t dst = tmem_base + Cfg::SF_COL0 + slot * Cfg::SLOT_COLS;
                        auto copy = [&](uint32_t col, uint32_t from) {
                            if constexpr (CG == 1) tmem_cp_32x128b_warpx4(dst + col, src + (from >> 4));
                            else tmem_cp_32x128b_warpx4_pair(dst + col, src + (from >> 4));
                        };
#pragma unroll
                        for (int c = 0; c < Cfg::CHUNKS; ++c) {
                            copy(4 * c, kScaleTile * c);
#pragma unroll
                            for (int b = 0; b < Cfg::Q_BLOCKS; ++b)
                                copy(4 * (Cfg::CHUNKS + Cfg::Q_BLOCKS * c + b), Cfg::SF_BYTES * (1 + b) + kScaleTile * c);
                        }
                        mma_commit<CG>(sf_full(slot), 0x1);
                    }
                    __syncwarp();
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            for (int i = 0; ok && i < Cfg::SF_SLOTS; ++i, ++n) {
                if (!mbar_wait_warp(sf_empty(n % Cfg::SF_SLOTS), ((n / Cfg::SF_SLOTS) & 1u) ^ 1u, abort_flag,
                                    2 * a.timeout_ns)) {
                    if (issue) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleSfCopy * 16 + kBarTail);
                    ok = false;
                }
            }
        }
    } else {
        // ----------------------------------------------------- epilogue --
        const uint32_t sub = warp & 3u;                         // TMEM lane quarter
        const int part = static_cast<int>(warp - Cfg::EPI0) / 4;
        constexpr int PARTS = Cfg::EPI_WARPS / 4;               // fours of warps that share a tile's rows of C
        constexpr int CHUNKS = Cfg::BQ / 32 / PARTS;            // of 32 rows, for each of them
        const Factor scale(Cfg::NV && a.ga ? __ldcg(a.ga) : 1.0f, Cfg::NV && a.gb ? __ldcg(a.gb) : 1.0f);
        const float alpha = scale.first;
        const int64_t esize = a.f32 ? 4 : 2;
        ColumnsOut to(base + Cfg::OUT_OFF, part, sub, lane, a.ldc * esize);
        const int mine = static_cast<int>(sub * 32u + lane);   // this lane's column
        uint32_t done = 0;
        const bool far = Cfg::NV && scale.second != 1.0f && members == 1;
        if (far)
            fp4_far_tiles<Cfg>(a, scale, tmem_base, tfull_bar(0), tempty_bar(0), abort_flag, abort_slot, first, step, rank);
        for (int tile = far ? num_tiles : first; tile < num_tiles; tile += step, ++done) {
            int tq, tp;
            raster_tile(tile, tiles_q, tiles_p, 8, tq, tp);
            const uint32_t buf = done % Cfg::ACC_BUFS;
            uint32_t ready = 1;
            if (lane == 0 && !mbar_wait(tfull_bar(buf), (done / Cfg::ACC_BUFS) & 1u, abort_flag, 3 * a.timeout_ns)) {
                record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleEpilogue * 16 + kBarTmemFull);
                ready = 0;
            }
            ready = __shfl_sync(0xFFFFFFFFu, ready, 0);
            if (!to.agree(ready != 0)) break;
            tc_fence_after_sync();
            const uint32_t acc = tmem_base + ((sub * 32u) << 16) + buf * Cfg::BQ;
            const int col0 = tp * Cfg::BP + static_cast<int>(rank) * Cfg::BP_CTA;
            const int count = min(Cfg::BQ, a.M - tq * Cfg::BQ);
            uint8_t *out = static_cast<uint8_t *>(a.c) + (static_cast<int64_t>(tq) * Cfg::BQ * a.ldc + col0) * esize;
            to.cols = a.N - col0;
            auto release = [&]() {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 1) mbar_arrive_local(tempty_bar(buf));
                    else mbar_arrive_cluster(map_to_cta(tempty_bar(buf), 0));
                }
            };
            if (Cfg::SPLIT && members > 1) {
                auto wait = [&]() {
                    if (mbar_wait_warp(received_bar, 0, abort_flag, 3 * a.timeout_ns)) return true;
                    if (lane == 0) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleEpilogue * 16 + kBarRxFull);
                    return false;
                };
                if (!cluster_sum(acc, mma_n(tq) / 4, static_cast<int>(members), static_cast<int>(me), sub * 32u + lane,
                                 base + Cfg::PART_OFF, received_bar, wait, out + mine * esize, to.ld_bytes, count,
                                 mine < to.cols, a.f32, scale))
                    break;
                release();
                continue;
            }
            // A single accumulator goes into registers whole, so that the next
            // tile's MMAs wait for that alone.
            constexpr int HELD = Cfg::ACC_BUFS == 1 ? CHUNKS : 1;
            if (a.f32) {
                float v[HELD][32];
#pragma unroll
                for (int chunk = 0; chunk < CHUNKS; ++chunk) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(acc + 32 * (chunk * PARTS + part), r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[chunk % HELD][i] = alpha * __uint_as_float(r[i]);
                    if (HELD > 1) continue;
                    const int j = 32 * (chunk * PARTS + part);
                    store_columns<32>(out + j * to.ld_bytes + mine * esize, to.ld_bytes, count - j, mine < to.cols, true,
                                      0.0f, v[0]);
                }
                release();
                if (HELD > 1)
#pragma unroll
                    for (int chunk = 0; chunk < CHUNKS; ++chunk) {
                        const int j = 32 * (chunk * PARTS + part);
                        store_columns<32>(out + j * to.ld_bytes + mine * esize, to.ld_bytes, count - j, mine < to.cols,
                                          true, 0.0f, v[chunk % HELD]);
                    }
            } else {
                uint32_t w[CHUNKS][16];
                load_chunks_bf16<CHUNKS>(acc + 32 * part, 32 * PARTS, alpha, w);
                release();
#pragma unroll
                for (int chunk = 0; chunk < CHUNKS; ++chunk) {
                    const int j = 32 * (chunk * PARTS + part);
                    if (j < count) to.rows(w[chunk], out + j * to.ld_bytes, count - j);
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (cluster > 1) cluster_sync_all();
    if (*abort_flag) {      // set in every CTA of the cluster before that; copies in flight land first
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 200000ull) __nanosleep(1000);
        __syncthreads();
        if (cluster > 1) cluster_sync_all();
    }
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<CG>(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace b200
