// Host side of the operators around the products (include/b200gemm.h): the
// RMS norm, the MXFP8 quantiser and the product with 4-bit weights.  Argument
// checks first, then one launch (two where a sum over rows needs its own).
// None of them keeps state, allocates or synchronises.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "b200gemm.h"
#include "gemm_w4_sm100.cuh"
#include "host.h"
#include "mxfp8_quantize_sm100.cuh"
#include "rmsnorm_sm100.cuh"

namespace {

using b200::kBF16;
using b200::kF32;
using b200::kNone;
using b200::host::aligned16;
using b200::host::extent_ok;
using b200::host::kMaxDim;
using b200::host::overlaps;
using b200::host::pitch16;

bool valid_type(gemm_out_t t) { return t == GEMM_OUT_F32 || t == GEMM_OUT_BF16; }
int64_t size_of(gemm_out_t t) { return t == GEMM_OUT_F32 ? 4 : 2; }

// One matrix of a call: rows x cols elements of `esize` bytes, pitch ld.
struct Mat {
    const void *p;
    int64_t rows, cols, ld, esize;
};

// Pointer, pitch, alignment and extent of a matrix that the call touches.
gemm_status_t check_mat(const Mat &m) {
    if (!m.p || m.ld < m.cols) return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(m.p) || !pitch16(m.ld, m.esize)) return GEMM_ERR_MISALIGNED;
    if (!extent_ok(m.rows, m.ld, m.esize)) return GEMM_ERR_TOO_LARGE;
    return GEMM_OK;
}

bool overlap(const Mat &a, const Mat &b) {
    return overlaps(a.p, a.rows, a.cols, a.ld, a.esize, b.p, b.rows, b.cols, b.ld, b.esize);
}

// The same matrix in the same place: element (i, j) of one is (i, j) of the other.
bool same(const Mat &a, const Mat &b) { return a.p == b.p && a.ld == b.ld && a.esize == b.esize; }

// A matrix that is written may overlap nothing else of the call.
template <size_t N>
bool any_overlap(const Mat &out, const Mat (&others)[N]) {
    for (const Mat &o : others)
        if (overlap(out, o)) return true;
    return false;
}

// One launch with programmatic dependence on the kernel before it in the
// stream (wait_for_stream in the kernels): its blocks take their places while
// that one finishes, which saves about a microsecond between two calls.
// cluster: blocks per cluster along x.
template <class... Params, class... Args>
gemm_status_t launch(void (*kernel)(Params...), dim3 grid, dim3 block, int smem, cudaStream_t stream, int cluster,
                     Args... args) {
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, kernel, static_cast<Params>(args)...);
    return e == cudaSuccess ? GEMM_OK : b200::host::cuda_fail(e);
}

// Dynamic shared memory that the blocks of an SM may take together (of its
// 228 KB, 1 KB per block is the system's, and static arrays count too).
constexpr int kSmemPerSm = 222 * 1024;

int round_up(int64_t n, int m) { return static_cast<int>((n + m - 1) / m * m); }

// ---------------------------------------------------------------- RMS norm --

// Threads per row and eights per thread.  Up to 1024 elements a warp holds the
// row, and eight rows share a block.  Longer rows take a block each: with
// fewer rows than would fill the SMs, one eight per thread (the shortest chain
// of loads); else four of bf16 or, with an fp32 operand, two, about the same
// bytes in flight.  Measured with four and with two, 4000 rows, bf16 out: fp32
// stream 12.7 and 11.3 us at 1100 elements, 25.7 and 24.2 at 3000, 61.8 and 59.8 at
// 8192; bf16 without a stream 7.2 and 5.9 at 1120, 12.9 and 12.7 at 3008, 21.5 and
// 23.0 at 6016, 26.7 and 30.3 at 8192; bf16 stream 10.7 and 8.6, 19.2 and 17.9, 33.4
// and 31.7, 42.8 and 41.6, but 75.2 and 79.4 with codes out at 8192 x 8192: for bf16
// four is the better one of long rows, and gives up to 20 % away on short ones.
// VPT 0: the row does not fit into registers.
struct RowShape {
    int vpt;
    dim3 block;
};

RowShape row_shape(int64_t K, bool few_rows, bool fp32) {
    const int64_t vecs = (K + 7) / 8;
    const auto block = [&](int vpt) { return dim3(static_cast<unsigned>(round_up((vecs + vpt - 1) / vpt, 32))); };
    if (vecs <= 128) return {vecs <= 32 ? 1 : vecs <= 64 ? 2 : 4, dim3(32, 8)};
    if (vecs <= 1024 && few_rows) return {1, block(1)};
    if (vecs <= 1024 && fp32) return {2, block(2)};
    if (vecs <= 2048) return {4, block(4)};
    return {0, dim3(1024)};
}

template <int XT, int HT, int VPT>
gemm_status_t launch_norm(int dev, const b200::RmsnormArgs &a, dim3 block, cudaStream_t stream) {
    const int64_t blocks = (a.M + block.y - 1) / block.y;
    gemm_status_t s;
    if constexpr (VPT == 0) {
        if ((s = b200::host::prepare<b200::rmsnorm_long_kernel<XT, HT>>(dev, 0, stream)) != GEMM_OK) return s;
        return launch(b200::rmsnorm_long_kernel<XT, HT>, dim3(static_cast<unsigned>(blocks)), block, 0, stream, 1, a);
    } else {
        if ((s = b200::host::prepare<b200::rmsnorm_kernel<XT, HT, VPT>>(dev, 0, stream)) != GEMM_OK) return s;
        return launch(b200::rmsnorm_kernel<XT, HT, VPT>, dim3(static_cast<unsigned>(blocks)), block, 0, stream, 1, a);
    }
}

template <int XT, int HT>
gemm_status_t dispatch_norm(int dev, int sm_count, const b200::RmsnormArgs &a, cudaStream_t stream) {
    const RowShape r = row_shape(a.K, a.M <= 2 * sm_count, XT == kF32 || HT == kF32);
    switch (r.vpt) {
        case 1: return launch_norm<XT, HT, 1>(dev, a, r.block, stream);
        case 2: return launch_norm<XT, HT, 2>(dev, a, r.block, stream);
        case 4: return launch_norm<XT, HT, 4>(dev, a, r.block, stream);
        default: return launch_norm<XT, HT, 0>(dev, a, r.block, stream);
    }
}

template <int XT>
gemm_status_t dispatch_norm_h(int dev, int sm_count, const b200::RmsnormArgs &a, int ht, cudaStream_t stream) {
    if (ht == kNone) return dispatch_norm<XT, kNone>(dev, sm_count, a, stream);
    return ht == kF32 ? dispatch_norm<XT, kF32>(dev, sm_count, a, stream)
                      : dispatch_norm<XT, kBF16>(dev, sm_count, a, stream);
}

// Rows of the backward pass's workspace, and so its blocks at most: a documented
// size that does not depend on the device.  A launch has one block per SM, 148 on
// this one.
constexpr int64_t kPartialRows = 296;
static_assert(kPartialRows <= 320, "rmsnorm_dw_kernel adds up to 320 shares");

// VPT 0: rows too long for registers.
template <int YT, int HT, int DT, int VPT>
gemm_status_t launch_back(int dev, int sm_count, b200::RmsnormBackArgs a, dim3 block, float *dw, float *ws,
                          cudaStream_t stream) {
    // One block per SM (its registers allow 512 threads): as many rows as that
    // holds at a time, and two to four in shared memory for each.
    const auto row_bytes = [&](bool stage_dr) {
        return static_cast<int>(VPT * 16 * block.x) * b200::back_pieces<YT, HT, DT>(stage_dr);
    };
    a.stage_dr = VPT < 4 || 2 * row_bytes(true) <= kSmemPerSm;
    if (VPT > 0) {
        const int64_t share = (a.M + sm_count - 1) / sm_count;      // rows per SM
        if (VPT < 4)    // with four eights per thread a row takes more than half of the threads
            block.y = static_cast<unsigned>(std::min<int64_t>({b200::kMaxRows, 512 / block.x, share,
                                                               kSmemPerSm / (2 * row_bytes(a.stage_dr))}));
        a.ring = std::min(4, kSmemPerSm / (row_bytes(a.stage_dr) * static_cast<int>(block.y)));
    }
    const int smem = a.ring * row_bytes(a.stage_dr) * static_cast<int>(block.y);
    const int64_t rows = (a.M + block.y - 1) / block.y;
    const int64_t blocks = std::min({rows, static_cast<int64_t>(sm_count), kPartialRows});
    const dim3 grid(static_cast<unsigned>(blocks));
    // one block's share of dw is dw itself
    if (dw) a.partial = blocks == 1 ? dw : ws;
    gemm_status_t s;
    if (dw && blocks > 1 && (s = b200::host::prepare<b200::rmsnorm_dw_kernel>(dev, 0, stream)) != GEMM_OK) return s;
    if constexpr (VPT == 0) {
        if ((s = b200::host::prepare<b200::rmsnorm_back_long_kernel<YT, HT, DT>>(dev, 0, stream)) != GEMM_OK) return s;
        s = launch(b200::rmsnorm_back_long_kernel<YT, HT, DT>, grid, block, 0, stream, 1, a);
    } else {
        if ((s = b200::host::prepare<b200::rmsnorm_back_kernel<YT, HT, DT, VPT>>(dev, kSmemPerSm, stream)) != GEMM_OK)
            return s;
        s = launch(b200::rmsnorm_back_kernel<YT, HT, DT, VPT>, grid, block, smem, stream, 1, a);
    }
    if (s != GEMM_OK || !dw || blocks == 1) return s;
    return launch(b200::rmsnorm_dw_kernel, dim3(static_cast<unsigned>((a.K + 31) / 32)), dim3(1024), 0, stream, 1, ws,
                  dw, blocks, a.K);
}

// One eight per thread up to 256 elements (a warp), two as far as 512 threads
// go (8192 elements), then four, as far as 512 threads go and shared memory holds
// two rows of dy and h (16384 elements; 13312 with both in fp32); past that two
// passes per row.  More than one eight spreads what a thread does once per row
// (addresses, the sum across the warps) over more elements (8000 x 1000 bf16: 18.9
// us with two, 25.7 with one, 23.3 with four in one warp).
template <int YT, int HT, int DT>
gemm_status_t dispatch_back(int dev, int sm_count, const b200::RmsnormBackArgs &a, float *dw, float *ws,
                            cudaStream_t stream) {
    const int64_t vecs = (a.K + 7) / 8;
    const auto block = [&](int vpt) { return dim3(static_cast<unsigned>(round_up((vecs + vpt - 1) / vpt, 32))); };
    if (vecs <= 32) return launch_back<YT, HT, DT, 1>(dev, sm_count, a, dim3(32), dw, ws, stream);
    if (vecs <= 1024) return launch_back<YT, HT, DT, 2>(dev, sm_count, a, block(2), dw, ws, stream);
    if (vecs <= 2048 && 2 * 16 * b200::back_pieces<YT, HT, DT>(false) * 4 * block(4).x <= kSmemPerSm)
        return launch_back<YT, HT, DT, 4>(dev, sm_count, a, block(4), dw, ws, stream);
    return launch_back<YT, HT, DT, 0>(dev, sm_count, a, dim3(1024), dw, ws, stream);
}

// --------------------------------------------------------- MXFP8 quantiser --

template <int XT, int VPT>
gemm_status_t launch_quantize_rows(int dev, const void *X, uint8_t *Q, uint8_t *sf, int64_t M, int64_t K, int64_t ldx,
                                   int64_t ldq, cudaStream_t stream) {
    const int64_t vecs = K / 8;
    dim3 block(32, 8);
    if (vecs > 32 * VPT) block = dim3(static_cast<unsigned>(std::min(256, round_up((vecs + VPT - 1) / VPT, 32))));
    const int64_t parts = (vecs + VPT * block.x - 1) / (VPT * block.x);
    const int64_t blocks = (M + block.y - 1) / block.y * parts;
    if (blocks > kMaxDim) return GEMM_ERR_TOO_LARGE;
    gemm_status_t s;
    if ((s = b200::host::prepare<b200::mx_quantize_kernel<XT, VPT>>(dev, 0, stream)) != GEMM_OK) return s;
    return launch(b200::mx_quantize_kernel<XT, VPT>, dim3(static_cast<unsigned>(blocks)), block, 0, stream, 1, X, Q, sf,
                  M, K, ldx, ldq, parts);
}

template <int XT>
gemm_status_t launch_quantize(int dev, int sm_count, const void *X, uint8_t *Q, uint8_t *sf, int64_t M, int64_t K,
                              int64_t ldx, int64_t ldq, gemm_layout_t layout, cudaStream_t stream) {
    gemm_status_t s;
    if (layout == GEMM_LAYOUT_MNMAJOR) {
        const int64_t i_tiles = (M + 63) / 64, blocks = i_tiles * ((K + 127) / 128);
        if (blocks > kMaxDim) return GEMM_ERR_TOO_LARGE;
        if ((s = b200::host::prepare<b200::mx_quantize_mn_kernel<XT>>(dev, 0, stream)) != GEMM_OK) return s;
        return launch(b200::mx_quantize_mn_kernel<XT>, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, stream, 1, X,
                      Q, sf, M, K, ldx, ldq, i_tiles);
    }
    // Four eights per thread; eight of bf16 where there are many rows: a block
    // then has as many bytes in flight as with fp32 (8192 x 8192 bf16: 34.2
    // against 35.6 us; 1000 x 8192: 4.9 against 4.7).
    if constexpr (XT == kBF16)
        if (M >= 16 * sm_count) return launch_quantize_rows<XT, 8>(dev, X, Q, sf, M, K, ldx, ldq, stream);
    return launch_quantize_rows<XT, 4>(dev, X, Q, sf, M, K, ldx, ldq, stream);
}

// ------------------------------------------------------- 4-bit weights --

// Blocks of a kernel that a device holds at once in clusters of 1, 2, 4 and 8:
// fewer for larger clusters, which the SMs of a GPC do not always fill (two
// blocks per SM: 296 of 148 SMs alone, but 284 in fours and 264 in eights).
// Asked once per kernel and device, before any capture.
struct ClusterRoom {
    std::atomic<int> blocks[b200::host::kMaxDevices][4];
};

template <class Cfg, int U>
gemm_status_t cluster_room(int dev, int sm_count, cudaStream_t stream, int (&room)[4]) {
    static ClusterRoom known{};
    gemm_status_t s;
    if ((s = b200::host::prepare<b200::gemm_w4_kernel<Cfg, U>>(dev, Cfg::SMEM_BYTES, stream)) != GEMM_OK) return s;
    for (int shift = 0; shift < 4; ++shift) {
        room[shift] = known.blocks[dev][shift].load(std::memory_order_relaxed);
        if (room[shift] > 0) continue;
        int n = Cfg::PER_SM * sm_count;
        if (shift > 0) {
            cudaLaunchConfig_t lc = {};
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 1u << shift;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            lc.gridDim = dim3(1024);
            lc.blockDim = dim3(Cfg::THREADS);
            lc.dynamicSmemBytes = Cfg::SMEM_BYTES;
            lc.attrs = &attr;
            lc.numAttrs = 1;
            int clusters = 0;
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters, b200::gemm_w4_kernel<Cfg, U>, &lc);
            if (e != cudaSuccess) return b200::host::cuda_fail(e);
            n = std::max(1, clusters << shift);
        }
        known.blocks[dev][shift].store(n, std::memory_order_relaxed);
        room[shift] = n;
    }
    return GEMM_OK;
}

template <class Cfg, int U>
gemm_status_t launch_w4(int dev, int sm_count, b200::W4Args a, cudaStream_t stream) {
    gemm_status_t s;
    int room[4];
    if ((s = cluster_room<Cfg, U>(dev, sm_count, stream, room)) != GEMM_OK) return s;
    const int64_t tiles = (a.N + Cfg::ROWS - 1) / Cfg::ROWS;
    const int64_t token_blocks = (a.M + 8 * Cfg::NT - 1) / (8 * Cfg::NT);
    const int64_t stages = (a.K + b200::kW4K - 1) / b200::kW4K;
    // K in 1, 2, 4 or 8 shares: as many as leave all blocks resident at once (a
    // second round of a few clusters took half as long again: 27.9 against
    // 19.2 us at 16 x 8192 x 8192 with 74 clusters of four)
    int shift = 0;
    while (shift < 3 && (tiles * token_blocks << (shift + 1)) <= room[shift + 1] && (int64_t(2) << shift) <= stages)
        ++shift;
    if (token_blocks > 65535 || tiles << shift > kMaxDim) return GEMM_ERR_TOO_LARGE;
    a.stages = static_cast<uint32_t>(stages);
    a.split_shift = shift;
    const dim3 grid(static_cast<unsigned>(tiles << shift), static_cast<unsigned>(token_blocks));
    return launch(b200::gemm_w4_kernel<Cfg, U>, grid, dim3(Cfg::THREADS), Cfg::SMEM_BYTES, stream, 1 << shift, a);
}

template <class Cfg>
gemm_status_t dispatch_w4(int dev, int sm_count, const b200::W4Args &a, cudaStream_t stream) {
    switch (a.group_shift) {
        case 5: return launch_w4<Cfg, 1>(dev, sm_count, a, stream);
        case 6: return launch_w4<Cfg, 2>(dev, sm_count, a, stream);
        case 7: return launch_w4<Cfg, 4>(dev, sm_count, a, stream);
        default: return launch_w4<Cfg, 8>(dev, sm_count, a, stream);
    }
}

gemm_status_t zero_rows(void *p, int64_t rows, int64_t cols, int64_t ld, int64_t esize, cudaStream_t stream) {
    const cudaError_t e = rows == 1 ? cudaMemsetAsync(p, 0, static_cast<size_t>(cols * esize), stream)
                                    : cudaMemset2DAsync(p, static_cast<size_t>(ld * esize), 0,
                                                        static_cast<size_t>(cols * esize), static_cast<size_t>(rows),
                                                        stream);
    return e == cudaSuccess ? GEMM_OK : b200::host::cuda_fail(e);
}

}  // namespace

extern "C" {

gemm_status_t gemm_rmsnorm(const void *X, const void *R, void *H, const float *weight, void *Y, uint8_t *Q, uint8_t *sf,
                           float *rstd, int64_t M, int64_t K, int64_t ldx, int64_t ldr, int64_t ldh, int64_t ldy,
                           int64_t ldq, gemm_out_t x_type, gemm_out_t h_type, float eps, cudaStream_t stream) {
    if (M < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M > kMaxDim || K > kMaxDim) return GEMM_ERR_TOO_LARGE;
    if (!valid_type(x_type) || (R && !valid_type(h_type)) || !(eps > 0.0f)) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || K == 0) return GEMM_OK;
    if (!X || !weight || (!Y && !Q) || (H && !R) || (Q && !sf)) return GEMM_ERR_INVALID_VALUE;
    if (Q && K % 32) return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(weight)) return GEMM_ERR_MISALIGNED;
    const Mat none{nullptr, 0, 0, 0, 1};
    const Mat mx{X, M, K, ldx, size_of(x_type)};
    const Mat mr = R ? Mat{R, M, K, ldr, size_of(h_type)} : none;
    const Mat mh = H ? Mat{H, M, K, ldh, size_of(h_type)} : none;
    const Mat my = Y ? Mat{Y, M, K, ldy, 2} : none;
    const Mat mq = Q ? Mat{Q, M, K, ldq, 1} : none;
    const Mat mw{weight, 1, K, K, 4};
    const Mat ms = Q ? Mat{sf, 1, M * (K / 32), M * (K / 32), 1} : none;
    const Mat mt = rstd ? Mat{rstd, 1, M, M, 4} : none;
    gemm_status_t s;
    for (const Mat *m : {&mx, &mr, &mh, &my, &mq})
        if (m->p && (s = check_mat(*m)) != GEMM_OK) return s;
    if (rstd && (reinterpret_cast<uintptr_t>(rstd) & 3u)) return GEMM_ERR_MISALIGNED;
    // outputs overlap nothing, except H, which may be R itself
    if (any_overlap(mh, {mx, same(mh, mr) ? none : mr, mw, my, mq, ms, mt}) ||
        any_overlap(my, {mx, mr, mw, mq, ms, mt}) || any_overlap(mq, {mx, mr, mw, ms, mt}) ||
        any_overlap(ms, {mx, mr, mw, mt}) || any_overlap(mt, {mx, mr, mw}))
        return GEMM_ERR_ALIAS;
    int dev, sm_count;
    if ((s = b200::host::device(dev, sm_count, stream)) != GEMM_OK) return s;
    const b200::RmsnormArgs a{X, R, H, weight, Y, Q, sf, rstd, M, K, ldx, ldr, ldh, ldy, ldq, eps};
    const int ht = !R ? kNone : h_type == GEMM_OUT_F32 ? kF32 : kBF16;
    return x_type == GEMM_OUT_F32 ? dispatch_norm_h<kF32>(dev, sm_count, a, ht, stream)
                                  : dispatch_norm_h<kBF16>(dev, sm_count, a, ht, stream);
}

int64_t gemm_rmsnorm_backward_workspace(int64_t M, int64_t K) {
    if (M <= 0 || K <= 0 || M > kMaxDim || K > kMaxDim) return 0;
    return std::min(M, kPartialRows) * K * 4;
}

gemm_status_t gemm_rmsnorm_backward(const void *dY, const void *H, const float *weight, const float *rstd, const void *dR,
                                    void *dH, float *dW, void *workspace, int64_t workspace_bytes, int64_t M, int64_t K,
                                    int64_t lddy, int64_t ldh, int64_t lddr, int64_t lddh, gemm_out_t dy_type,
                                    gemm_out_t h_type, gemm_out_t dh_type, cudaStream_t stream) {
    if (M < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M > kMaxDim || K > kMaxDim) return GEMM_ERR_TOO_LARGE;
    if (!valid_type(dy_type) || !valid_type(h_type) || !valid_type(dh_type)) return GEMM_ERR_INVALID_VALUE;
    if (K == 0) return GEMM_OK;
    gemm_status_t s;
    int dev, sm_count;
    const Mat none{nullptr, 0, 0, 0, 1};
    if (dW && !aligned16(dW)) return GEMM_ERR_MISALIGNED;
    if (M == 0) {   // the empty sum
        if (!dW) return GEMM_OK;
        if ((s = b200::host::device(dev, sm_count, stream)) != GEMM_OK) return s;
        return zero_rows(dW, 1, K, K, 4, stream);
    }
    if (!dY || !H || !weight || !rstd || !dH) return GEMM_ERR_INVALID_VALUE;
    const int64_t need = dW ? gemm_rmsnorm_backward_workspace(M, K) : 0;
    if (dW && (!workspace || workspace_bytes < need)) return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(weight) || (dW && !aligned16(workspace)) || (reinterpret_cast<uintptr_t>(rstd) & 3u))
        return GEMM_ERR_MISALIGNED;
    const Mat my{dY, M, K, lddy, size_of(dy_type)};
    const Mat mh{H, M, K, ldh, size_of(h_type)};
    const Mat mr = dR ? Mat{dR, M, K, lddr, size_of(dh_type)} : none;
    const Mat md{dH, M, K, lddh, size_of(dh_type)};
    const Mat mw{weight, 1, K, K, 4};
    const Mat mt{rstd, 1, M, M, 4};
    const Mat mg = dW ? Mat{dW, 1, K, K, 4} : none;
    const Mat mp = dW ? Mat{workspace, 1, need, need, 1} : none;
    for (const Mat *m : {&my, &mh, &mr, &md})
        if (m->p && (s = check_mat(*m)) != GEMM_OK) return s;
    // outputs overlap nothing, except dH, which may be dY or dR itself
    if (any_overlap(md, {same(md, my) ? none : my, same(md, mr) ? none : mr, mh, mw, mt, mg, mp}) ||
        any_overlap(mg, {my, mh, mr, mw, mt, mp}) || any_overlap(mp, {my, mh, mr, mw, mt}))
        return GEMM_ERR_ALIAS;
    if ((s = b200::host::device(dev, sm_count, stream)) != GEMM_OK) return s;
    const b200::RmsnormBackArgs a{dY, H, weight, rstd, dR, dH, nullptr, M, K, lddy, ldh, lddr, lddh, 0,
                                  1.0f / static_cast<float>(K), true};
    float *ws = static_cast<float *>(workspace);
    const auto f32 = [](gemm_out_t t) { return t == GEMM_OUT_F32 ? 1 : 0; };
    switch (4 * f32(dy_type) + 2 * f32(h_type) + f32(dh_type)) {
        case 0: return dispatch_back<kBF16, kBF16, kBF16>(dev, sm_count, a, dW, ws, stream);
        case 1: return dispatch_back<kBF16, kBF16, kF32>(dev, sm_count, a, dW, ws, stream);
        case 2: return dispatch_back<kBF16, kF32, kBF16>(dev, sm_count, a, dW, ws, stream);
        case 3: return dispatch_back<kBF16, kF32, kF32>(dev, sm_count, a, dW, ws, stream);
        case 4: return dispatch_back<kF32, kBF16, kBF16>(dev, sm_count, a, dW, ws, stream);
        case 5: return dispatch_back<kF32, kBF16, kF32>(dev, sm_count, a, dW, ws, stream);
        case 6: return dispatch_back<kF32, kF32, kBF16>(dev, sm_count, a, dW, ws, stream);
        default: return dispatch_back<kF32, kF32, kF32>(dev, sm_count, a, dW, ws, stream);
    }
}

gemm_status_t gemm_mxfp8_quantize(const void *X, uint8_t *Q, uint8_t *sf, int64_t M, int64_t K, int64_t ldx, int64_t ldq,
                                  gemm_out_t x_type, gemm_layout_t layout, cudaStream_t stream) {
    if (M < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M > kMaxDim || K > kMaxDim) return GEMM_ERR_TOO_LARGE;
    if (!valid_type(x_type) || (layout != GEMM_LAYOUT_KMAJOR && layout != GEMM_LAYOUT_MNMAJOR) || K % 32)
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || K == 0) return GEMM_OK;
    if (!X || !Q || !sf) return GEMM_ERR_INVALID_VALUE;
    const bool mn = layout == GEMM_LAYOUT_MNMAJOR;
    const Mat mx{X, mn ? K : M, mn ? M : K, ldx, size_of(x_type)};
    const Mat mq{Q, M, K, ldq, 1};
    const Mat ms{sf, 1, M * (K / 32), M * (K / 32), 1};
    gemm_status_t s;
    if ((s = check_mat(mx)) != GEMM_OK || (s = check_mat(mq)) != GEMM_OK) return s;
    if (overlap(mq, mx) || overlap(mq, ms) || overlap(ms, mx)) return GEMM_ERR_ALIAS;
    int dev, sm_count;
    if ((s = b200::host::device(dev, sm_count, stream)) != GEMM_OK) return s;
    return x_type == GEMM_OUT_F32 ? launch_quantize<kF32>(dev, sm_count, X, Q, sf, M, K, ldx, ldq, layout, stream)
                                  : launch_quantize<kBF16>(dev, sm_count, X, Q, sf, M, K, ldx, ldq, layout, stream);
}

gemm_status_t gemm_bf16_w4(const void *A, const uint8_t *B, const void *scales, const uint8_t *zeros, void *C, int64_t M,
                           int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t lds, int64_t ldc, int64_t group,
                           gemm_out_t c_type, cudaStream_t stream) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return GEMM_ERR_TOO_LARGE;
    if (!valid_type(c_type) || K % 32 || group < 32 || (group & (group - 1))) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return GEMM_OK;
    const int64_t ec = size_of(c_type);
    const Mat mc{C, M, N, ldc, ec};
    gemm_status_t s;
    if ((s = check_mat(mc)) != GEMM_OK) return s;
    int dev, sm_count;
    if (K == 0) {   // the empty sum
        if ((s = b200::host::device(dev, sm_count, stream)) != GEMM_OK) return s;
        return zero_rows(C, M, N, ldc, ec, stream);
    }
    const int64_t groups = (K + group - 1) / group;
    const Mat ma{A, M, K, lda, 2};
    const Mat mb{B, N, K / 2, ldb, 1};
    const Mat ms{scales, N, groups, lds, 2};
    const Mat mz{zeros, N, groups, lds, 1};
    for (const Mat *m : {&ma, &mb, &ms, &mz})
        if ((m != &mz || zeros) && (s = check_mat(*m)) != GEMM_OK) return s;
    if (lds % 16) return GEMM_ERR_MISALIGNED;   // rows of zeros too, whether given or not
    if (any_overlap(mc, {ma, mb, ms, mz})) return GEMM_ERR_ALIAS;
    if ((s = b200::host::device(dev, sm_count, stream)) != GEMM_OK) return s;
    int shift = 5;
    while ((int64_t(1) << shift) < group && shift < 31) ++shift;   // K < 2^31: one group either way from there
    b200::W4Args a{};
    a.a = static_cast<const uint16_t *>(A);
    a.b = B;
    a.scales = static_cast<const uint16_t *>(scales);
    a.zeros = zeros;
    a.c = C;
    a.M = M, a.N = N, a.K = K, a.lda = lda, a.ldb = ldb, a.lds = lds, a.ldc = ldc;
    a.groups = groups;
    a.group_shift = shift;
    a.out = c_type == GEMM_OUT_F32 ? kF32 : kBF16;
    // A kernel for each size of batch: its sums stay in registers, its activations
    // pass through shared memory.  Up to 32 rows two blocks share an SM, with as
    // many ring stages as their shared memory allows; from 33 rows on the sums'
    // registers leave room for one block, which takes about half of it.
    if (M <= 8) return dispatch_w4<b200::W4Cfg<1, 8, 4>>(dev, sm_count, a, stream);
    if (M <= 16) return dispatch_w4<b200::W4Cfg<2, 8, 3>>(dev, sm_count, a, stream);
    if (M <= 24) return dispatch_w4<b200::W4Cfg<3, 8, 3>>(dev, sm_count, a, stream);
    if (M <= 32) return dispatch_w4<b200::W4Cfg<4, 8, 2>>(dev, sm_count, a, stream);
    if (M <= 48) return dispatch_w4<b200::W4Cfg<6, 8, 3>>(dev, sm_count, a, stream);
    return dispatch_w4<b200::W4Cfg<8, 8, 2>>(dev, sm_count, a, stream);
}

}  // extern "C"
