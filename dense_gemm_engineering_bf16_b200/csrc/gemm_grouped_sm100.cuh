// Products grouped by expert, on rows sorted by expert whose extents only the
// device knows (ends[e]: where expert e's rows end):
//
//   rows       C[r] = A[r] . B_e            for the rows r of expert e
//   gradient   dB_e = sum over its rows r of dC[r]^T A[r]   (+ beta dB_e)
//
// One persistent, warp-specialised kernel with two operands: P, whose index runs
// along a row of the output and along the MMA's M (128 a CTA, TMEM lanes), and
// Q, whose index runs along its columns and the MMA's N.  N is chosen per tile
// in the instruction descriptor, in steps of 16 (32 for a pair of CTAs), so the
// ragged side costs what it has: an expert with 300 rows is two tiles of 150
// (160), one with three rows a tile of 16.
//   rows       P = B_e (rows of N, K- or MN-major), Q = A, reduced over K
//   gradient   P, Q = A, dC or the other way round, both MN-major, reduced over
//              the expert's rows
//
// Warps of a CTA:
//   0          TMA producer
//   1          MMA issuer (of the pair's leader), owner of TMEM
//   2          gradient only: an expert's last block of 64 rows ends inside rows
//              of the next expert, which must not count, not even as 0 * NaN.
//              Such a block's bytes arrive on a barrier of its own; this warp
//              zeroes the foreign rows up to the MMA's next step of 16 in both
//              operands and hands the block on.
//   the rest   epilogue: TMEM to registers to global memory (columns_out.cuh),
//              which overlaps the next tile's MMAs
//
// SPLIT, for the few rows of a token: a cluster of 2, 4 or 8 CTAs owns a tile,
// each over a share of K, and their partials meet in distributed shared memory
// (cluster_sum).  One tile per cluster.  A share is one accumulator's sum, so
// with an fp32 result no longer than a segment: K of about 1024, 2048 or 4096.
//
// Every CTA works out the tiles from `ends` itself: the numbers of tiles up to
// each expert in shared memory, a binary search per tile.  Rows outside every
// expert are neither computed nor written.
//
// What bounds it (one B200, in bursts; runs of many seconds are held by the
// power limit to 1.2 to 1.6 GHz of 1.97 and take up to a quarter longer):
//   large experts  the tensor pipe and its power: 16384 x 4096 x 2048 in one group
//                  185 to 194 us (1.4 to 1.5 PFLOP/s), in 32 of different sizes 218
//                  to 232 (tensor pipe 80 % busy, every weight read once; narrower
//                  tiles load P more often for the same work)
//   few rows each  memory: 128 rows on 64 experts of 2048 x 4096, 740 MB in 125 us,
//                  92 % of the copy rate
//   one token      the start and the end (3.4 us without any work; a pair of CTAs 6)
//                  and the ramp between: 2 of 8 experts of 4096 x 2048, 33.6 MB,
//                  10.9 us
//   gradient       the write-back, of 256 x 256 values for each few blocks of MMAs:
//                  32 experts, 512 rows each, 4096 x 2048, bf16 261 us, of which the
//                  stores are 41 and taking the accumulators out 44 (218 without the
//                  operands' loads); 64 experts, 256 rows each 401 us, stores 74,
//                  accumulators 129 (371 without loads).  8 experts, 1000 rows, 1024 x
//                  512, fp32: 8.2 us
// The pairs' rows kernels spill 44 bytes a thread, at the 168 registers that 320
// threads leave.
#pragma once
#include <climits>
#include <cstdint>

#include "columns_out.cuh"
#include "gemm_bf16_sm100.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace b200 {

constexpr int kMaxGroups = 1024;      // three words of shared memory each

// What a kernel computes: rows of C, or an expert's gradient.
enum : int { kGroupedRows = 0, kGroupedGrad = 1 };

template <int MODE_, bool PMN_, int CG_, int BQ_, int STAGES_, bool SPLIT_ = false>
struct GroupedCfg {
    static constexpr int MODE = MODE_;
    static constexpr bool SPLIT = SPLIT_;
    static constexpr bool PMN = PMN_ || MODE_ == kGroupedGrad;   // P stored MN-major
    static constexpr bool QMN = MODE_ == kGroupedGrad;
    static constexpr int CG = CG_;
    static constexpr int BP_CTA = 128;               // P indexes (TMEM lanes) per CTA
    static constexpr int BP = BP_CTA * CG;
    static constexpr int BQ = BQ_;                   // largest Q extent of a tile
    static constexpr int STAGES = STAGES_;
    static constexpr int BK = 64;
    static constexpr int N_STEP = 16 * CG;           // MMA N is a multiple of this
    static constexpr int Q_CTA = BQ / CG;            // Q indexes this CTA loads at most
    static constexpr int QBOX = QMN ? 64 : BQ >= 128 ? 32 : 16;   // Q indexes per TMA box
    static constexpr int P_BYTES = BP_CTA * BK * 2;
    static constexpr int Q_BYTES = Q_CTA * BK * 2;
    static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
    static constexpr int EPI_WARPS = BQ >= 128 ? 8 : 4;
    static constexpr int EPI0 = MODE == kGroupedGrad ? 3 : 2;    // first epilogue warp
    static constexpr int THREADS = 32 * (EPI0 + EPI_WARPS);
    // full[S], empty[S], tmem_full[2], tmem_empty[2], fix[S] (gradient), received (split)
    static constexpr int NUM_BARS = (MODE == kGroupedGrad ? 3 : 2) * STAGES + 4 + (SPLIT ? 1 : 0);
    static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
    static constexpr int OUT_OFF = BAR_OFF + (NUM_BARS * 8 + 8 + 127) / 128 * 128;    // + TMEM address, abort flag
    static constexpr int PART_OFF = OUT_OFF + EPI_WARPS / 4 * kOutBytes;      // other members' partials
    static constexpr int TABLE_OFF = PART_OFF + (SPLIT ? BQ * 128 * 4 : 0);
    static constexpr int TMEM_COLS = pow2_at_least(2 * BQ, 32);
    static constexpr int smem_bytes(int groups) { return 1024 + TABLE_OFF + 12 * groups; }

    static_assert(Q_CTA % QBOX == 0 && Q_BYTES % 1024 == 0, "whole boxes and swizzle atoms");
    static_assert(BQ >= 32 && BQ <= 256, "the epilogue reads 32 columns at a time");
    static_assert(!SPLIT || (CG == 1 && EPI_WARPS == 4 && MODE == kGroupedRows), "split: one-CTA tiles of rows");
    static_assert(smem_bytes(kMaxGroups) <= 232448, "dynamic shared memory per CTA on sm_100");
    // wait_for_stream lets the next kernel's blocks come while TMEM is still being
    // allocated here: one that allocates as well may not fit beside this one
    static_assert(smem_bytes(0) > 233472 / 2, "more than half of an SM's shared memory");
};

struct GroupedArgs {
    const int32_t *ends;
    void *out;
    int64_t ld, out_stride;     // of the output; gradient: between experts
    int groups, M;              // rows of A and of dC
    int P, Q, K;                // P's extent (columns of the output); gradient: Q's (its rows); rows: K
    float beta;                 // gradient
    bool f32;                   // type of the output
    int segment;                // blocks of the reduction that the tensor core sums by itself (a split's share: all)
    DeviceStatus *status;
    uint64_t timeout_ns;
};

// One tile: P indexes from p0, Q indexes [q0, q0 + count) (rows: of A and C;
// gradient: rows of the output), `n` the MMA's N, reduction from k0 over k_len.
struct GroupedTile {
    int group, p0, q0, count, n, k0, k_len;

    // for the warps that issue copies and MMAs
    __device__ __forceinline__ GroupedTile uniform() const {
        return {b200::uniform(group), b200::uniform(p0), b200::uniform(q0), b200::uniform(count), b200::uniform(n),
                b200::uniform(k0), b200::uniform(k_len)};
    }
};

// Where the tiles are, the same in every warp: one look-up per tile and role,
// so it has no division but these (a dozen of them were 1000 cycles a tile).
template <class Cfg>
struct GroupedTiles {
    const int *ends, *tiles, *widths;   // shared memory; gradient: ends alone
    int groups, P, Q, k0, k_len;        // rows: this CTA's share of K
    int tiles_p, tiles_q, width;        // gradient: tiles along Q, and their width
    Divisor band, per;                  // tiles of eight Q tiles' band; of a group (gradient)

    __device__ __forceinline__ static int width_of(int extent) {
        return parts_of(parts_of(extent, max(parts_of(extent, Cfg::BQ), 1)), Cfg::N_STEP) * Cfg::N_STEP;
    }

    __device__ __forceinline__ GroupedTiles(const GroupedArgs &a, const int *ends_, const int *tiles_, const int *widths_,
                                            int members, int me)
        : ends(ends_), tiles(tiles_), widths(widths_), groups(a.groups), P(a.P), Q(a.Q), k0(0), k_len(a.K),
          tiles_p(parts_of(a.P, Cfg::BP)), tiles_q(parts_of(a.Q, Cfg::BQ)), width(width_of(a.Q)),
          band(8 * static_cast<uint32_t>(tiles_p)), per(static_cast<uint32_t>(max(tiles_p * tiles_q, 1))) {
        if (members > 1) {
            const int64_t blocks = (int64_t(a.K) + Cfg::BK - 1) / Cfg::BK;
            k0 = static_cast<int>(blocks * me / members * Cfg::BK);
            // the last share's end may be 2^31
            k_len = static_cast<int>(min(blocks * (me + 1) / members * Cfg::BK, static_cast<int64_t>(a.K)) - k0);
        }
    }

    __device__ __forceinline__ int count() const {
        return Cfg::MODE == kGroupedGrad ? groups * tiles_p * tiles_q : tiles[groups - 1];
    }

    __device__ __forceinline__ GroupedTile operator()(int tile) const {
        GroupedTile t;
        int local, extent, n, wide;     // Q tiles, of `wide` (the last may be smaller)
        if constexpr (Cfg::MODE == kGroupedRows) {
            int lo = 0, hi = groups - 1;      // the first group whose tiles reach past `tile`
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (tiles[mid] > tile) hi = mid;
                else lo = mid + 1;
            }
            t.group = lo;
            local = tile - (lo ? tiles[lo - 1] : 0);
            t.q0 = lo ? ends[lo - 1] : 0;
            extent = ends[lo] - t.q0;
            n = parts_of(extent, Cfg::BQ);
            wide = widths[lo];
            t.k0 = k0;
            t.k_len = k_len;
        } else {
            t.group = static_cast<int>(per.divide(tile));
            local = tile - t.group * tiles_p * tiles_q;
            t.q0 = 0;
            extent = Q;
            n = tiles_q;
            wide = width;
            t.k0 = t.group ? ends[t.group - 1] : 0;
            t.k_len = ends[t.group] - t.k0;
        }
        // bands of eight Q tiles, so that clusters running at the same time
        // share both operands in L2
        const int b = static_cast<int>(band.divide(local)), in_band = local - b * 8 * tiles_p, rows = min(n - 8 * b, 8);
        const int tp = static_cast<int>(divide_small(in_band, rows)), tq = 8 * b + in_band - tp * rows;
        t.p0 = tp * Cfg::BP;
        t.q0 += tq * wide;
        t.count = min(wide, extent - tq * wide);
        t.n = parts_of(t.count, Cfg::N_STEP) * Cfg::N_STEP;
        return t;
    }
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
gemm_grouped_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ, GroupedArgs a) {
    constexpr int CG = Cfg::CG, STAGES = Cfg::STAGES;
    constexpr bool GRAD = Cfg::MODE == kGroupedGrad;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t base = smem_addr(smem);
    const uint32_t warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const uint32_t rank = CG == 2 ? cluster_cta_rank() : 0u;
    const int members = Cfg::SPLIT ? static_cast<int>(cluster_num_ctas()) : 1;
    const int me = Cfg::SPLIT ? static_cast<int>(cluster_cta_rank()) : 0;
    const int cluster = CG * members;

    const uint32_t bar0 = base + Cfg::BAR_OFF;
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
    auto fix_bar = [&](uint32_t s) { return bar0 + 8u * (2 * STAGES + 4 + s); };
    const uint32_t received_bar = bar0 + 8u * (Cfg::NUM_BARS - 1);
    const uint32_t tmem_slot = bar0 + 8u * Cfg::NUM_BARS, abort_slot = tmem_slot + 4u;
    volatile uint32_t *tmem_slot_ptr = reinterpret_cast<volatile uint32_t *>(smem + Cfg::BAR_OFF + 8 * Cfg::NUM_BARS);
    volatile uint32_t *abort_flag = tmem_slot_ptr + 1;
    int *ends = reinterpret_cast<int *>(smem + Cfg::TABLE_OFF), *tiles = ends + a.groups, *widths = tiles + a.groups;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            // gradient: each CTA of the pair says that its part of a block is there
            mbar_init(full_bar(s), GRAD ? CG : 1);
            mbar_init(empty_bar(s), 1);
            if (GRAD) mbar_init(fix_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), Cfg::EPI_WARPS * CG);
        }
        if (Cfg::SPLIT) mbar_init(received_bar, 128 * max(members - 1, 1));
        *abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc<CG>(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish<CG>();
    }
    wait_for_stream();
    // from L2: the kernel before may have written them while this block was already here
    for (int e = threadIdx.x; e < a.groups; e += Cfg::THREADS) ends[e] = min(max(__ldcg(a.ends + e), 0), a.M);
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        // An end below an earlier one counts as that one, so that the experts'
        // rows never overlap; then the tiles up to each expert's last.
        const int tiles_p = parts_of(a.P, Cfg::BP);
        int top = 0, before = 0;
        for (int e0 = 0; e0 < a.groups; e0 += 32) {
            const int e = e0 + static_cast<int>(lane);
            int end = e < a.groups ? ends[e] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, end, d);
                if (static_cast<int>(lane) >= d) end = max(end, up);
            }
            end = max(end, top);
            int start = __shfl_up_sync(0xFFFFFFFFu, end, 1);
            if (lane == 0) start = top;
            top = __shfl_sync(0xFFFFFFFFu, end, 31);
            int n = 0;
            if (e < a.groups) {
                ends[e] = end;
                n = parts_of(end - start, Cfg::BQ) * tiles_p;
                widths[e] = GroupedTiles<Cfg>::width_of(end - start);
            }
            if constexpr (!GRAD) {
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int up = __shfl_up_sync(0xFFFFFFFFu, n, d);
                    if (static_cast<int>(lane) >= d) n += up;
                }
                if (e < a.groups) tiles[e] = before + n;
                before += __shfl_sync(0xFFFFFFFFu, n, 31);
            }
        }
    }
    __syncthreads();
    if (cluster > 1) cluster_sync_all();
    tc_fence_after_sync();
    const uint32_t tmem_base = static_cast<uint32_t>(uniform(static_cast<int>(*tmem_slot_ptr)));
    const GroupedTiles<Cfg> tile_at(a, ends, tiles, widths, members, me);
    const int num_tiles = tile_at.count();
    const int first = static_cast<int>(blockIdx.x) / cluster, step = static_cast<int>(gridDim.x) / cluster;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer --
        const bool issue = elect_one();
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        for (int tile = first; ok && tile < num_tiles; tile += step) {
            const GroupedTile t = tile_at(tile).uniform();
            const int p = t.p0 + static_cast<int>(rank) * Cfg::BP_CTA;
            const int q_cta = t.n / CG, q = t.q0 + static_cast<int>(rank) * q_cta;
            const int boxes = (q_cta + Cfg::QBOX - 1) / Cfg::QBOX;
            const uint32_t bytes = Cfg::P_BYTES + boxes * Cfg::QBOX * Cfg::BK * 2;
            for (int left = t.k_len; left > 0; left -= Cfg::BK) {
                const int k = t.k0 + (t.k_len - left);
                if (!mbar_wait_warp(empty_bar(stage), phase ^ 1u, abort_flag, 2 * a.timeout_ns)) {
                    if (issue) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleProducer * 16 + kBarEmpty);
                    ok = false;
                    break;
                }
                const uint32_t p_dst = base + stage * Cfg::STAGE_BYTES, q_dst = p_dst + Cfg::P_BYTES;
                if (GRAD && left < Cfg::BK && left % 16 != 0) {     // through warp 2
                    if (issue) {
                        const uint32_t bar = fix_bar(stage);
                        mbar_arrive_expect_tx(bar, bytes);
                        tma_load_2d(p_dst, &tmP, bar, p, k);
                        tma_load_2d(p_dst + 8192u, &tmP, bar, p + 64, k);
                        for (int b = 0; b < boxes; ++b) tma_load_2d(q_dst + 8192u * b, &tmQ, bar, q + 64 * b, k);
                    }
                } else if (issue) {
                    // bytes are counted by the pair's leader
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), CG * bytes);
                    else if (GRAD) mbar_arrive_cluster_relaxed(map_to_cta(full_bar(stage), 0));
                    const uint32_t bar = CG == 2 ? map_to_cta(full_bar(stage), 0) : full_bar(stage);
                    auto load2 = [&](uint32_t dst, const CUtensorMap *m, int x, int y) {
                        if constexpr (CG == 1) tma_load_2d(dst, m, bar, x, y);
                        else tma_load_2d_pair(dst, m, bar, x, y);
                    };
                    auto load3 = [&](uint32_t dst, const CUtensorMap *m, int x, int y, int z) {
                        if constexpr (CG == 1) tma_load_3d(dst, m, bar, x, y, z);
                        else tma_load_3d_pair(dst, m, bar, x, y, z);
                    };
                    if constexpr (GRAD) {
                        load2(p_dst, &tmP, p, k);
                        load2(p_dst + 8192u, &tmP, p + 64, k);
                        for (int b = 0; b < boxes; ++b) load2(q_dst + 8192u * b, &tmQ, q + 64 * b, k);
                    } else {
                        if constexpr (Cfg::PMN) {
                            load3(p_dst, &tmP, p, k, t.group);
                            load3(p_dst + 8192u, &tmP, p + 64, k, t.group);
                        } else {
                            load3(p_dst, &tmP, k, p, t.group);
                        }
                        for (int b = 0; b < boxes; ++b) load2(q_dst + Cfg::QBOX * 128u * b, &tmQ, k, q + Cfg::QBOX * b);
                    }
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
            // Descriptors of stage 0, step 0; a stage and a step of 16 add their
            // offset to the address field, one add per operand and MMA.
            const uint64_t p_desc0 = operand_desc(base, 0, Cfg::PMN), q_desc0 = operand_desc(base + Cfg::P_BYTES, 0, Cfg::QMN);
            constexpr uint32_t p_step = (Cfg::PMN ? 2048u : 32u) >> 4, q_step = (Cfg::QMN ? 2048u : 32u) >> 4;
            const bool issue = elect_one();
            uint32_t stage = 0, phase = 0, done = 0;
            bool ok = true;
            for (int tile = first; ok && tile < num_tiles; tile += step) {
                const GroupedTile t = tile_at(tile).uniform();
                const uint32_t idesc = idesc_bf16_f32(Cfg::BP, t.n, Cfg::PMN, Cfg::QMN);
                int until = 0;          // blocks until the segment's end
                uint32_t acc = 0, more = 0;
                for (int left = t.k_len; left > 0; left -= Cfg::BK) {
                    if (until == 0) {
                        const uint32_t buf = done & 1u;
                        if (!mbar_wait_warp(tempty_bar(buf), ((done >> 1) & 1u) ^ 1u, abort_flag, 3 * a.timeout_ns)) {
                            if (issue) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleMma * 16 + kBarTmemEmpty);
                            ok = false;
                            break;
                        }
                        acc = tmem_base + buf * Cfg::BQ;
                        more = 0;
                        until = members > 1 ? INT_MAX : a.segment;
                    }
                    if (!mbar_wait_warp(full_bar(stage), phase, abort_flag, a.timeout_ns)) {
                        if (issue) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleMma * 16 + kBarFull);
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const bool last = --until == 0 || left <= Cfg::BK;
                    if (issue) {
                        const uint64_t p_desc = p_desc0 + (stage * Cfg::STAGE_BYTES >> 4);
                        const uint64_t q_desc = q_desc0 + (stage * Cfg::STAGE_BYTES >> 4);
                        mma_bf16_ss<CG>(acc, p_desc, q_desc, idesc, more);
                        if (left >= Cfg::BK) {
#pragma unroll
                            for (int j = 1; j < Cfg::BK / 16; ++j)
                                mma_bf16_ss<CG>(acc, p_desc + j * p_step, q_desc + j * q_step, idesc, 1u);
                        } else {
                            for (int j = 1; 16 * j < left; ++j)
                                mma_bf16_ss<CG>(acc, p_desc + j * p_step, q_desc + j * q_step, idesc, 1u);
                        }
                        mma_commit<CG>(empty_bar(stage), 0x3);
                        if (last) mma_commit<CG>(tfull_bar(done & 1u), 0x3);
                    }
                    __syncwarp();
                    more = 1;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (last) {
                        ++done;
                        until = 0;
                    }
                }
            }
        }
    } else if (GRAD && warp == 2) {
        // ------------------------- rows of the next expert in a last block --
        uint32_t blocks = 0, parity = 0;       // blocks so far; bit s: parity of fix[s]
        for (int tile = first; tile < num_tiles; tile += step) {
            const GroupedTile t = tile_at(tile);
            blocks += parts_of(t.k_len, Cfg::BK);
            if (t.k_len % 16 == 0) continue;
            const uint32_t stage = (blocks - 1) % STAGES;
            if (!mbar_wait_warp(fix_bar(stage), (parity >> stage) & 1u, abort_flag, 3 * a.timeout_ns)) {
                if (lane == 0) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleFix * 16 + kBarFix);
                break;
            }
            parity ^= 1u << stage;
            // a row of a box is 128 bytes, swizzled within itself
            const int used = t.k_len % Cfg::BK, clear = (16 - used % 16) * 128;
            const int boxes = 2 + (t.n / CG + 63) / 64;         // P's, then Q's, 8 KB apart
            uint8_t *at = smem + stage * Cfg::STAGE_BYTES + used * 128;
            for (int b = 0; b < boxes; ++b)
                for (int i = 16 * static_cast<int>(lane); i < clear; i += 512)
                    *reinterpret_cast<uint4 *>(at + 8192 * b + i) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2) mbar_arrive_cluster(map_to_cta(full_bar(stage), 0));
                else mbar_arrive_local(full_bar(stage));
            }
        }
        __syncwarp();
    } else {
        // ----------------------------------------------------- epilogue --
        const uint32_t sub = warp & 3u;                         // TMEM lane quarter
        const int part = static_cast<int>(warp - Cfg::EPI0) / 4;
        constexpr int PARTS = Cfg::EPI_WARPS / 4;               // fours of warps that share a tile's rows of the output
        constexpr int CHUNKS = Cfg::BQ / 32 / PARTS;            // of 32 rows, for each of them
        const int64_t esize = a.f32 ? 4 : 2;
        ColumnsOut to(base + Cfg::OUT_OFF, part, sub, lane, a.ld * esize);
        uint32_t done = 0;
        // the accumulator of a tile's next segment is complete
        auto wait_full = [&]() {
            const bool ready = mbar_wait_warp(tfull_bar(done & 1u), (done >> 1) & 1u, abort_flag, 3 * a.timeout_ns);
            if (!ready && lane == 0) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleEpilogue * 16 + kBarTmemFull);
            tc_fence_after_sync();
            return ready;
        };
        auto release = [&]() {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (CG == 1) mbar_arrive_local(tempty_bar(done & 1u));
                else mbar_arrive_cluster(map_to_cta(tempty_bar(done & 1u), 0));
            }
            ++done;
        };
        for (int tile = first; tile < num_tiles; tile += step) {
            const GroupedTile t = tile_at(tile);
            const int col0 = t.p0 + static_cast<int>(rank) * Cfg::BP_CTA;
            uint8_t *out = static_cast<uint8_t *>(a.out) + col0 * esize +
                           ((GRAD ? t.group * a.out_stride : 0) + static_cast<int64_t>(t.q0) * a.ld) * esize;
            to.cols = a.P - col0;
            auto from = [&](int chunk) {
                return tmem_base + ((sub * 32u) << 16) + (done & 1u) * Cfg::BQ + 32u * (chunk * PARTS + part);
            };
            if (Cfg::SPLIT && members > 1) {
                auto wait = [&]() {
                    if (mbar_wait_warp(received_bar, 0, abort_flag, 3 * a.timeout_ns)) return true;
                    if (lane == 0) record_timeout(a.status, abort_flag, abort_slot, cluster, kRoleEpilogue * 16 + kBarRxFull);
                    return false;
                };
                const int c = static_cast<int>(sub * 32u + lane);
                if (!wait_full() || !cluster_sum(from(0), t.n / 4, members, me, c, base + Cfg::PART_OFF, received_bar, wait,
                                                 out + c * esize, to.ld_bytes, t.count, c < to.cols, a.f32, Factor(1.0f, 1.0f)))
                    break;
                release();
                continue;
            }
            // one segment whose sum is only rounded; otherwise sums go through registers in fp32
            const bool packed = !a.f32 && (!GRAD || a.beta == 0.0f) && t.k_len <= a.segment * Cfg::BK;
            if (packed) {
                if (!to.agree(t.k_len == 0 || wait_full())) break;
                uint32_t w[CHUNKS][16] = {};
                if (t.k_len > 0) {
                    load_chunks_bf16<CHUNKS>(from(0), 32 * PARTS, 1.0f, w);
                    release();
                }
#pragma unroll
                for (int chunk = 0; chunk < CHUNKS; ++chunk) {
                    const int j = 32 * (chunk * PARTS + part);
                    if (j < t.count) to.rows(w[chunk], out + j * to.ld_bytes, t.count - j);
                }
                continue;
            }
            // The tensor core cuts what its sums do not hold, always towards zero, so
            // the error grows with the length (4.5e-6 of an fp32 result at 4096);
            // segments are added here, to nearest (5e-7)
            float v[CHUNKS][32] = {};
            bool ok = true;
            for (int left = t.k_len; left > 0 && ok; left -= a.segment * Cfg::BK) {
                ok = wait_full();
                if (!ok) break;
#pragma unroll
                for (int chunk = 0; chunk < CHUNKS; ++chunk) {
                    if (32 * (chunk * PARTS + part) < t.count) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(from(chunk), r);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[chunk][i] += __uint_as_float(r[i]);
                    }
                }
                release();
            }
            if (!ok) break;
            const int c = static_cast<int>(sub * 32u + lane);
#pragma unroll
            for (int chunk = 0; chunk < CHUNKS; ++chunk) {
                const int j = 32 * (chunk * PARTS + part);
                if (j < t.count)
                    store_columns<32>(out + j * to.ld_bytes + c * esize, to.ld_bytes, t.count - j, c < to.cols, a.f32,
                                      GRAD ? a.beta : 0.0f, v[chunk]);
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
