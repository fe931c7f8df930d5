// Host side of the products that leave the dense bf16 path (include/b200gemm.h):
// grouped by expert, and of 4-bit floating-point operands with their
// quantiser.  Argument checks first, then one launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "b200gemm.h"
#include "fp4_quantize_sm100.cuh"
#include "gemm_fp4_sm100.cuh"
#include "gemm_grouped_sm100.cuh"
#include "host.h"

namespace {

using b200::DeviceStatus;
using b200::host::aligned16;
using b200::host::extent_ok;
using b200::host::kMaxDim;
using b200::host::overlaps;
using b200::host::pitch16;

bool valid_type(gemm_out_t t) { return t == GEMM_OUT_F32 || t == GEMM_OUT_BF16; }
bool valid_format(gemm_fp4_t f) { return f == GEMM_FP4_MX || f == GEMM_FP4_NV; }
bool valid_layout(gemm_layout_t l) { return l == GEMM_LAYOUT_KMAJOR || l == GEMM_LAYOUT_MNMAJOR; }
int64_t size_of(gemm_out_t t) { return t == GEMM_OUT_F32 ? 4 : 2; }

// `count` matrices of a call, `stride` elements apart: rows x cols elements of
// `esize` bytes, pitch ld.
struct Mat {
    const void *p;
    int64_t rows, cols, ld, esize, count = 1, stride = 0;
    // elements from the first of a matrix to its last
    int64_t span() const { return (rows - 1) * ld + cols; }
};

// Pointer, pitch, alignment and extent; several matrices may not overlap.
gemm_status_t check_mat(const Mat &m) {
    if (!m.p || m.ld < m.cols) return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(m.p) || !pitch16(m.ld, m.esize)) return GEMM_ERR_MISALIGNED;
    if (!extent_ok(m.rows, m.ld, m.esize)) return GEMM_ERR_TOO_LARGE;
    if (m.count > 1) {
        if (m.stride < m.span()) return GEMM_ERR_INVALID_VALUE;
        if (!pitch16(m.stride, m.esize)) return GEMM_ERR_MISALIGNED;
        if (!extent_ok(m.count, m.stride, m.esize)) return GEMM_ERR_TOO_LARGE;
    }
    return GEMM_OK;
}

bool overlap(const Mat &a, const Mat &b) {
    return overlaps(a.p, a.count, a.span(), a.stride, a.esize, b.p, b.count, b.span(), b.stride, b.esize);
}

// Clusters of `size` blocks of a kernel that a device holds at once, possibly
// none.  Asked once per kernel, device and size, before any capture.
template <auto Kernel>
gemm_status_t resident_clusters(int dev, int sm_count, int threads, int smem, int size, int &n, cudaStream_t stream) {
    static std::atomic<int> known[b200::host::kMaxDevices][4];      // one more than the answer
    const int slot = size >= 8 ? 3 : size >= 4 ? 2 : size >= 2 ? 1 : 0;
    n = known[dev][slot].load(std::memory_order_relaxed) - 1;
    if (n >= 0) return GEMM_OK;
    if (b200::host::capturing(stream)) return GEMM_ERR_CAPTURE;
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(size);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    lc.gridDim = dim3(static_cast<unsigned>(sm_count / size * size));
    lc.blockDim = dim3(static_cast<unsigned>(threads));
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    lc.attrs = &attr;
    lc.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, Kernel, &lc);
    if (e != cudaSuccess) return b200::host::cuda_fail(e);
    known[dev][slot].store(n + 1, std::memory_order_relaxed);
    return GEMM_OK;
}

// One launch in clusters of `size` blocks, with programmatic dependence on the
// kernel before it in the stream (wait_for_stream in the kernels).
template <class... Params, class... Args>
gemm_status_t launch(void (*kernel)(Params...), int clusters, int size, int threads, int smem, cudaStream_t stream,
                     const Args &...args) {
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(size);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    lc.gridDim = dim3(static_cast<unsigned>(clusters * size));
    lc.blockDim = dim3(static_cast<unsigned>(threads));
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&lc, kernel, args...);
    return e == cudaSuccess ? GEMM_OK : b200::host::cuda_fail(e);
}

template <class... Params, class... Args>
gemm_status_t launch(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.stream = stream;
    lc.attrs = &attr;
    lc.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, kernel, args...);
    return e == cudaSuccess ? GEMM_OK : b200::host::cuda_fail(e);
}

// ------------------------------------------------------ grouped by expert --

// K-major operand of bf16: rows of K, boxes of 64 x `box` rows.
gemm_status_t map_rows(CUtensorMap *map, const Mat &m, uint32_t box) {
    const int64_t dims[2] = {m.cols, m.rows}, strides[1] = {m.ld * 2};
    const uint32_t b[2] = {64, box};
    return b200::host::encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, m.p, 2, dims, strides, b,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// The experts' matrices: boxes of 64 x `box` rows of one of them.
gemm_status_t map_experts(CUtensorMap *map, const Mat &m, uint32_t box) {
    const int64_t stride = m.count > 1 ? m.stride : m.ld;     // one matrix: not looked at
    const int64_t dims[3] = {m.cols, m.rows, m.count}, strides[2] = {m.ld * 2, stride * 2};
    const uint32_t b[3] = {64, box, 1};
    return b200::host::encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, m.p, 3, dims, strides, b,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// Blocks of 64 that a tensor core sums by itself (gemm_grouped_kernel's epilogue):
// 512 elements for an fp32 result; 2^20 for a bf16 one, whose 2^16 MMAs take off
// 2^15 last places of the sum, 2^-8 of it, at the very most: half a step of bf16.
int segment_blocks(bool f32) { return f32 ? 8 : 1 << 14; }

constexpr int64_t kMaxTiles = int64_t(1) << 30;     // tile numbers are 32-bit, one grid's step on top

template <class Cfg>
gemm_status_t launch_grouped(int dev, int sm_count, const CUtensorMap &tmP, const CUtensorMap &tmQ,
                             const b200::GroupedArgs &a, int64_t tiles, cudaStream_t stream) {
    constexpr auto kernel = b200::gemm_grouped_kernel<Cfg>;
    constexpr int kMost = Cfg::smem_bytes(b200::kMaxGroups);
    if (tiles > kMaxTiles) return GEMM_ERR_TOO_LARGE;
    gemm_status_t s;
    int size = Cfg::CG, room;
    if ((s = b200::host::prepare<kernel>(dev, kMost, stream)) != GEMM_OK) return s;
    if constexpr (Cfg::SPLIT) {
        // K in as many shares as keep every cluster resident at once, eight blocks
        // of 64 each at least; for an fp32 result no longer than a segment
        const int64_t blocks = (int64_t(a.K) + Cfg::BK - 1) / Cfg::BK;
        for (size = 8; size > 1; size /= 2) {
            if ((s = resident_clusters<kernel>(dev, sm_count, Cfg::THREADS, kMost, size, room, stream)) != GEMM_OK) return s;
            if (tiles <= room && blocks >= 8 * size && (!a.f32 || (blocks + size - 1) / size <= a.segment)) break;
        }
    }
    if ((s = resident_clusters<kernel>(dev, sm_count, Cfg::THREADS, kMost, size, room, stream)) != GEMM_OK) return s;
    return launch(kernel, static_cast<int>(std::min<int64_t>(std::max(room, 1), tiles)), size, Cfg::THREADS,
                  Cfg::smem_bytes(a.groups), stream, tmP, tmQ, a);
}

template <class Cfg>
gemm_status_t launch_rows(int dev, int sm_count, const Mat &A, const Mat &B, const b200::GroupedArgs &a,
                          cudaStream_t stream) {
    alignas(64) CUtensorMap tmP{}, tmQ{};
    gemm_status_t s;
    if (a.K > 0) {
        if ((s = map_experts(&tmP, B, Cfg::PMN ? Cfg::BK : Cfg::BP_CTA)) != GEMM_OK) return s;
        if ((s = map_rows(&tmQ, A, Cfg::QBOX)) != GEMM_OK) return s;
    }
    // at most: whole tiles of all rows, and one more per expert that has rows
    const int64_t tiles = (a.M / Cfg::BQ + std::min(a.groups, a.M)) * ((int64_t(a.P) + Cfg::BP - 1) / Cfg::BP);
    return launch_grouped<Cfg>(dev, sm_count, tmP, tmQ, a, tiles, stream);
}

// Waves of `tiles` on `slots` of them at once.
double waves(double tiles, int slots) { return std::ceil(tiles / slots); }

// Tiles of `size` rows that experts with `rows` rows each on average take:
// their sizes differ, so about half a tile more than the average alone would.
double tiles_of(double experts, double rows, int size) {
    return experts > 1 ? experts * (rows / size + 0.5) : std::ceil(rows / size);
}

template <bool PMN>
gemm_status_t dispatch_rows(int dev, int sm_count, const Mat &A, const Mat &B, const b200::GroupedArgs &a,
                            cudaStream_t stream) {
    // Tiles of 64 rows for few rows an expert, or for tiles so few that K is
    // split (for an fp32 result where launch_grouped can).  Then single CTAs of 128 x 128 or pairs of 256 x 256, whichever is
    // predicted faster: a fixed cost, and per wave one of its own and one per 64
    // of K, in us (K = 2048, N = 2048, skewed, 64-row tiles, single, pair: 8 experts,
    // 64 rows 15.1 15.1 16.6; 512 rows 21.0 16.5 18.0; 4000 rows 60 40 37; 64 experts,
    // 2000 rows 89 93 90; 8000 rows 166 120 111.  One expert, 512 rows, K = 4096, N =
    // 512: 14.1 18.0 24.2).
    const int experts = std::min(a.groups, a.M);
    const double rows = static_cast<double>(a.M) / experts;
    const int64_t blocks = (int64_t(a.K) + 63) / 64, narrow = (int64_t(a.P) + 127) / 128, wide = (int64_t(a.P) + 255) / 256;
    if (rows <= 32 || (blocks >= 32 && 2 * (a.M / 64 + experts) * narrow <= sm_count))
        return launch_rows<b200::GroupedCfg<b200::kGroupedRows, PMN, 1, 64, 6, true>>(dev, sm_count, A, B, a, stream);
    const double one = 2.5 + waves(tiles_of(experts, rows, 128) * narrow, sm_count) * (1.0 + 0.226 * blocks);
    const double two = 5.0 + waves(tiles_of(experts, rows, 256) * wide, sm_count / 2) * (1.5 + 0.285 * blocks);
    if (one < two) return launch_rows<b200::GroupedCfg<b200::kGroupedRows, PMN, 1, 128, 5>>(dev, sm_count, A, B, a, stream);
    return launch_rows<b200::GroupedCfg<b200::kGroupedRows, PMN, 2, 256, 5>>(dev, sm_count, A, B, a, stream);
}

template <class Cfg>
gemm_status_t launch_grad(int dev, int sm_count, const Mat &p, const Mat &q, const b200::GroupedArgs &a,
                          cudaStream_t stream) {
    alignas(64) CUtensorMap tmP{}, tmQ{};
    gemm_status_t s;
    if (a.M > 0 && ((s = map_rows(&tmP, p, Cfg::BK)) != GEMM_OK || (s = map_rows(&tmQ, q, Cfg::BK)) != GEMM_OK)) return s;
    const int64_t tiles = ((p.cols + Cfg::BP - 1) / Cfg::BP) * ((q.cols + Cfg::BQ - 1) / Cfg::BQ);
    if (tiles > kMaxTiles) return GEMM_ERR_TOO_LARGE;
    return launch_grouped<Cfg>(dev, sm_count, tmP, tmQ, a, tiles * a.groups, stream);
}

gemm_status_t dispatch_grad(int dev, int sm_count, const Mat &p, const Mat &q, const b200::GroupedArgs &a,
                            cudaStream_t stream) {
    // As above, single CTAs of 128 x 128 or pairs of 256 x 256 (single, pair: 8
    // experts, 1000 rows, 1024 x 512 8.2 and 10.6 us; one, 8192 rows, 1024 x 1024 36
    // and 46, 2048 x 2048 69 and 54).
    const double tiles1 = static_cast<double>((p.cols + 127) / 128) * ((q.cols + 127) / 128) * a.groups;
    const double tiles2 = static_cast<double>((p.cols + 255) / 256) * ((q.cols + 255) / 256) * a.groups;
    const double blocks = std::ceil(static_cast<double>(a.M) / a.groups / 64);
    const double one = 2.5 + waves(tiles1, sm_count) * (1.2 + 0.252 * blocks);
    const double two = 4.5 + waves(tiles2, sm_count / 2) * (2.0 + 0.311 * blocks);
    if (one < two) return launch_grad<b200::GroupedCfg<b200::kGroupedGrad, true, 1, 128, 5>>(dev, sm_count, p, q, a, stream);
    return launch_grad<b200::GroupedCfg<b200::kGroupedGrad, true, 2, 256, 5>>(dev, sm_count, p, q, a, stream);
}

// ----------------------------------------------------------------- 4 bits --

int64_t block_of(gemm_fp4_t f) { return f == GEMM_FP4_NV ? b200::kFp4Block<true> : b200::kFp4Block<false>; }

// Scale tiles along K, and of a matrix.
int64_t scale_tiles_k(int64_t K, gemm_fp4_t f) { return (K + 4 * block_of(f) - 1) / (4 * block_of(f)); }
int64_t scale_tiles(int64_t rows, int64_t K, gemm_fp4_t f) { return (rows + 127) / 128 * scale_tiles_k(K, f); }

// Of a matrix's scales: 32-bit words in tiles, `chunks` neighbouring ones a box.
gemm_status_t map_scales(CUtensorMap *map, const uint8_t *sf, int64_t tiles, int chunks) {
    const int64_t dims[2] = {b200::kScaleTile / 4, tiles}, strides[1] = {b200::kScaleTile};
    const uint32_t b[2] = {b200::kScaleTile / 4, static_cast<uint32_t>(chunks)};
    return b200::host::encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, sf, 2, dims, strides, b,
                                  CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Codes: rows of bytes, boxes of 128 x `box` rows.
gemm_status_t map_codes(CUtensorMap *map, const Mat &m, uint32_t box) {
    const int64_t dims[2] = {m.cols, m.rows}, strides[1] = {m.ld};
    const uint32_t b[2] = {128, box};
    return b200::host::encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.p, 2, dims, strides, b,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
}

struct Fp4Call {
    Mat a, b;
    const uint8_t *sfa, *sfb;
    gemm_fp4_t format;
    b200::GemmFp4Args args;
};

template <class Cfg>
gemm_status_t launch_fp4(int dev, int sm_count, const Fp4Call &c, cudaStream_t stream) {
    constexpr auto kernel = b200::gemm_fp4_kernel<Cfg>;
    const int64_t tiles = ((int64_t(c.args.N) + Cfg::BP - 1) / Cfg::BP) * ((int64_t(c.args.M) + Cfg::BQ - 1) / Cfg::BQ);
    if (tiles > kMaxTiles || (Cfg::ONE_TILE_M && c.args.M > Cfg::BQ)) return GEMM_ERR_TOO_LARGE;
    gemm_status_t s;
    if ((s = b200::host::prepare<kernel>(dev, Cfg::SMEM_BYTES, stream)) != GEMM_OK) return s;
    int size = Cfg::CG, room;
    if constexpr (Cfg::SPLIT) {
        // K in as many shares as keep every cluster resident at once, two stages each at least
        const int64_t blocks = (int64_t(c.args.K) + Cfg::BK - 1) / Cfg::BK;
        for (size = 8; size > 1; size /= 2) {
            if ((s = resident_clusters<kernel>(dev, sm_count, Cfg::THREADS, Cfg::SMEM_BYTES, size, room, stream)) != GEMM_OK)
                return s;
            if (tiles <= room && blocks >= 2 * size) break;
        }
    }
    if ((s = resident_clusters<kernel>(dev, sm_count, Cfg::THREADS, Cfg::SMEM_BYTES, size, room, stream)) != GEMM_OK)
        return s;
    alignas(64) CUtensorMap tmP, tmQ, tmSP, tmSQ;
    if ((s = map_codes(&tmP, c.b, Cfg::BP_CTA)) != GEMM_OK || (s = map_codes(&tmQ, c.a, Cfg::QBOX)) != GEMM_OK ||
        (s = map_scales(&tmSP, c.sfb, scale_tiles(c.args.N, c.args.K, c.format), Cfg::CHUNKS)) != GEMM_OK ||
        (s = map_scales(&tmSQ, c.sfa, scale_tiles(c.args.M, c.args.K, c.format), Cfg::CHUNKS)) != GEMM_OK)
        return s;
    return launch(kernel, static_cast<int>(std::min<int64_t>(std::max(room, 1), tiles)), size, Cfg::THREADS, Cfg::SMEM_BYTES, stream,
                  tmP, tmQ, tmSP, tmSQ, c.args);
}

template <bool NV>
gemm_status_t dispatch_fp4(int dev, int sm_count, const Fp4Call &c, cudaStream_t stream) {
    // Up to 64 rows K is split over clusters.
    if (c.args.M <= 64) return launch_fp4<b200::GemmFp4Cfg<NV, 1, 64, 6, true>>(dev, sm_count, c, stream);
    // From there single CTAs of 128 x 128 or pairs of 256 x 256, whichever is
    // predicted faster: a fixed cost (pairs take 2.5 us longer to start and end),
    // and per wave one of its own and one per 256 of K, in us.  Measured, single
    // and pair: 1000 x 2048 x 2048 6.3 and 8.5, 512 x 4096 x 4096 8.8 and 10.8, 400
    // x 8192 x 8192 24.3 and 17.9, 1000 x 2500 x 2016 11.2 and 10.1.
    const double single = static_cast<double>((int64_t(c.args.M) + 127) / 128 * ((int64_t(c.args.N) + 127) / 128));
    const double pairs = static_cast<double>((int64_t(c.args.M) + 255) / 256 * ((int64_t(c.args.N) + 255) / 256));
    const double steps = static_cast<double>((int64_t(c.args.K) + 255) / 256);
    const double one = 2.3 + waves(single, sm_count) * (1.0 + 0.345 * steps);
    const double two = 4.8 + waves(pairs, sm_count / 2) * (0.8 + 0.36 * steps);
    if (two < one) return launch_fp4<b200::GemmFp4Cfg<NV, 2, 256, 5>>(dev, sm_count, c, stream);
    return launch_fp4<b200::GemmFp4Cfg<NV, 1, 128, 5>>(dev, sm_count, c, stream);
}

template <int XT, bool NV, int VPT, bool WIDE>
gemm_status_t launch_fp4_rows(int dev, const b200::Fp4QuantizeArgs &a, cudaStream_t stream) {
    const int64_t sixteens = a.K / 16, most = VPT == 1 ? 64 : 256;
    dim3 block(32, 8);
    if (sixteens > 32 * VPT)
        block = dim3(static_cast<unsigned>(std::min(most, ((sixteens + VPT - 1) / VPT + 31) / 32 * 32)));
    const int64_t parts = (sixteens + VPT * block.x - 1) / (VPT * block.x);
    const int64_t blocks = (a.M + block.y - 1) / block.y * parts;
    if (blocks > kMaxDim) return GEMM_ERR_TOO_LARGE;
    gemm_status_t s;
    if ((s = b200::host::prepare<b200::fp4_quantize_kernel<XT, NV, VPT, WIDE>>(dev, 0, stream)) != GEMM_OK) return s;
    return launch(b200::fp4_quantize_kernel<XT, NV, VPT, WIDE>, dim3(static_cast<unsigned>(blocks)), block, stream, a,
                  static_cast<unsigned>(parts));
}

template <int XT, bool NV>
gemm_status_t launch_fp4_quantize(int dev, int sm_count, const b200::Fp4QuantizeArgs &a, gemm_layout_t layout, cudaStream_t stream) {
    gemm_status_t s;
    if (layout == GEMM_LAYOUT_MNMAJOR) {
        const int64_t i_tiles = (a.M + 63) / 64, blocks = i_tiles * ((a.K + 127) / 128);
        if (blocks > kMaxDim) return GEMM_ERR_TOO_LARGE;
        if ((s = b200::host::prepare<b200::fp4_quantize_mn_kernel<XT, NV>>(dev, 0, stream)) != GEMM_OK) return s;
        return launch(b200::fp4_quantize_mn_kernel<XT, NV>, dim3(static_cast<unsigned>(blocks)), dim3(128), stream, a,
                      static_cast<unsigned>(i_tiles));
    }
    // Few rows: one sixteen per thread, in small blocks, so that a row spreads
    // over SMs; else four of bf16 or two of fp32, as many bytes in flight.
    const bool few = a.M * a.K <= int64_t(16) * 256 * sm_count;
    const bool wide = (reinterpret_cast<uintptr_t>(a.x) & 31u) == 0 && a.ldx * b200::elem_bytes<XT> % 32 == 0;
    if (few) return wide ? launch_fp4_rows<XT, NV, 1, true>(dev, a, stream) : launch_fp4_rows<XT, NV, 1, false>(dev, a, stream);
    constexpr int VPT = XT == b200::kF32 ? 2 : 4;
    return wide ? launch_fp4_rows<XT, NV, VPT, true>(dev, a, stream) : launch_fp4_rows<XT, NV, VPT, false>(dev, a, stream);
}

}  // namespace

extern "C" {

gemm_status_t gemm_bf16_grouped(const void *A, const void *B, const int32_t *ends, void *C, int64_t groups, int64_t M,
                                int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t strideb, int64_t ldc,
                                gemm_out_t c_type, gemm_layout_t b_layout, cudaStream_t stream) {
    if (groups < 0 || M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim || groups > b200::kMaxGroups) return GEMM_ERR_TOO_LARGE;
    if (!valid_type(c_type) || !valid_layout(b_layout)) return GEMM_ERR_INVALID_VALUE;
    if (groups == 0 || M == 0 || N == 0) return GEMM_OK;
    if (!ends) return GEMM_ERR_INVALID_VALUE;
    if (reinterpret_cast<uintptr_t>(ends) & 3u) return GEMM_ERR_MISALIGNED;
    const bool mn = b_layout == GEMM_LAYOUT_MNMAJOR;
    const Mat mc{C, M, N, ldc, size_of(c_type)};
    const Mat me{ends, 1, groups, groups, 4};
    const Mat ma{A, M, K, lda, 2};
    const Mat mb{B, mn ? K : N, mn ? N : K, ldb, 2, groups, strideb};
    gemm_status_t s;
    if ((s = check_mat(mc)) != GEMM_OK) return s;
    if (overlap(mc, me)) return GEMM_ERR_ALIAS;
    if (K > 0) {
        if ((s = check_mat(ma)) != GEMM_OK || (s = check_mat(mb)) != GEMM_OK) return s;
        if (overlap(mc, ma) || overlap(mc, mb)) return GEMM_ERR_ALIAS;
    }
    int dev, sm_count;
    DeviceStatus *status;
    if ((s = b200::host::device_with_status(dev, sm_count, status, stream)) != GEMM_OK) return s;
    b200::GroupedArgs a{};
    a.ends = ends;
    a.out = C;
    a.ld = ldc;
    a.groups = static_cast<int>(groups);
    a.M = static_cast<int>(M);
    a.P = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.f32 = c_type == GEMM_OUT_F32;
    a.segment = segment_blocks(a.f32);
    a.status = status;
    a.timeout_ns = b200::host::watchdog_ns(K);
    return mn ? dispatch_rows<true>(dev, sm_count, ma, mb, a, stream)
              : dispatch_rows<false>(dev, sm_count, ma, mb, a, stream);
}

gemm_status_t gemm_bf16_grouped_wgrad(const void *dC, const void *A, const int32_t *ends, void *dB, int64_t groups,
                                      int64_t M, int64_t N, int64_t K, int64_t lddc, int64_t lda, int64_t lddb,
                                      int64_t stridedb, gemm_out_t db_type, gemm_layout_t db_layout, float beta,
                                      cudaStream_t stream) {
    if (groups < 0 || M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim || groups > b200::kMaxGroups) return GEMM_ERR_TOO_LARGE;
    if (!valid_type(db_type) || !valid_layout(db_layout)) return GEMM_ERR_INVALID_VALUE;
    if (groups == 0 || N == 0 || K == 0) return GEMM_OK;
    if (!ends) return GEMM_ERR_INVALID_VALUE;
    if (reinterpret_cast<uintptr_t>(ends) & 3u) return GEMM_ERR_MISALIGNED;
    const bool mn = db_layout == GEMM_LAYOUT_MNMAJOR;
    const Mat mg{dB, mn ? K : N, mn ? N : K, lddb, size_of(db_type), groups, stridedb};
    const Mat me{ends, 1, groups, groups, 4};
    const Mat mc{dC, M, N, lddc, 2};
    const Mat ma{A, M, K, lda, 2};
    gemm_status_t s;
    if ((s = check_mat(mg)) != GEMM_OK) return s;
    if (overlap(mg, me)) return GEMM_ERR_ALIAS;
    if (M > 0) {
        if ((s = check_mat(mc)) != GEMM_OK || (s = check_mat(ma)) != GEMM_OK) return s;
        if (overlap(mg, mc) || overlap(mg, ma)) return GEMM_ERR_ALIAS;
    }
    int dev, sm_count;
    DeviceStatus *status;
    if ((s = b200::host::device_with_status(dev, sm_count, status, stream)) != GEMM_OK) return s;
    const Mat &p = mn ? mc : ma, &q = mn ? ma : mc;     // P's index runs along a row of dB
    b200::GroupedArgs a{};
    a.ends = ends;
    a.out = dB;
    a.ld = lddb;
    a.out_stride = stridedb;
    a.groups = static_cast<int>(groups);
    a.M = static_cast<int>(M);
    a.P = static_cast<int>(p.cols);
    a.Q = static_cast<int>(q.cols);
    a.beta = beta;
    a.f32 = db_type == GEMM_OUT_F32;
    a.segment = segment_blocks(a.f32);
    a.status = status;
    a.timeout_ns = b200::host::watchdog_ns(M);
    return dispatch_grad(dev, sm_count, p, q, a, stream);
}

int64_t gemm_fp4_scale_bytes(int64_t rows, int64_t K, gemm_fp4_t format) {
    if (rows <= 0 || K <= 0 || rows > kMaxDim || K > kMaxDim || !valid_format(format)) return 0;
    return scale_tiles(rows, K, format) * b200::kScaleTile;
}

gemm_status_t gemm_fp4_quantize(const void *X, const float *scale, uint8_t *Q, uint8_t *sf, int64_t M, int64_t K,
                                int64_t ldx, int64_t ldq, gemm_fp4_t format, gemm_out_t x_type, gemm_layout_t layout,
                                cudaStream_t stream) {
    if (M < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M > kMaxDim || K > kMaxDim) return GEMM_ERR_TOO_LARGE;
    if (!valid_type(x_type) || !valid_layout(layout) || !valid_format(format) || K % 32) return GEMM_ERR_INVALID_VALUE;
    if (format == GEMM_FP4_MX && scale) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || K == 0) return GEMM_OK;
    if (!X || !Q || !sf) return GEMM_ERR_INVALID_VALUE;
    const bool mn = layout == GEMM_LAYOUT_MNMAJOR;
    const int64_t sf_bytes = gemm_fp4_scale_bytes(M, K, format);
    const Mat mx{X, mn ? K : M, mn ? M : K, ldx, size_of(x_type)};
    const Mat mq{Q, M, K / 2, ldq, 1};
    const Mat ms{sf, 1, sf_bytes, sf_bytes, 1};
    const Mat mg{scale, 1, 1, 1, 4};
    gemm_status_t s;
    if ((s = check_mat(mx)) != GEMM_OK || (s = check_mat(mq)) != GEMM_OK) return s;
    if (!aligned16(sf) || (reinterpret_cast<uintptr_t>(scale) & 3u)) return GEMM_ERR_MISALIGNED;
    if (overlap(mq, mx) || overlap(mq, ms) || overlap(ms, mx) || overlap(mq, mg) || overlap(ms, mg)) return GEMM_ERR_ALIAS;
    int dev, sm_count;
    if ((s = b200::host::device(dev, sm_count, stream)) != GEMM_OK) return s;
    const b200::Fp4QuantizeArgs a{X, scale, Q, sf, M, K, ldx, ldq, scale_tiles_k(K, format)};
    if (format == GEMM_FP4_NV)
        return x_type == GEMM_OUT_F32 ? launch_fp4_quantize<b200::kF32, true>(dev, sm_count, a, layout, stream)
                                      : launch_fp4_quantize<b200::kBF16, true>(dev, sm_count, a, layout, stream);
    return x_type == GEMM_OUT_F32 ? launch_fp4_quantize<b200::kF32, false>(dev, sm_count, a, layout, stream)
                                  : launch_fp4_quantize<b200::kBF16, false>(dev, sm_count, a, layout, stream);
}

gemm_status_t gemm_fp4(const uint8_t *A, const uint8_t *sfa, const float *scale_a, const uint8_t *B, const uint8_t *sfb,
                       const float *scale_b, void *C, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                       int64_t ldc, gemm_fp4_t format, gemm_out_t c_type, cudaStream_t stream) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_VALUE;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return GEMM_ERR_TOO_LARGE;
    if (!valid_type(c_type) || !valid_format(format) || K % 32) return GEMM_ERR_INVALID_VALUE;
    if (format == GEMM_FP4_MX && (scale_a || scale_b)) return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return GEMM_OK;
    const int64_t ec = size_of(c_type);
    const Mat mc{C, M, N, ldc, ec};
    gemm_status_t s;
    if ((s = check_mat(mc)) != GEMM_OK) return s;
    int dev, sm_count;
    if (K == 0) {   // the empty sum
        if ((s = b200::host::device(dev, sm_count, stream)) != GEMM_OK) return s;
        const cudaError_t e = M == 1 ? cudaMemsetAsync(C, 0, static_cast<size_t>(N * ec), stream)
                                     : cudaMemset2DAsync(C, static_cast<size_t>(ldc * ec), 0, static_cast<size_t>(N * ec),
                                                         static_cast<size_t>(M), stream);
        return e == cudaSuccess ? GEMM_OK : b200::host::cuda_fail(e);
    }
    const Mat ma{A, M, K / 2, lda, 1}, mb{B, N, K / 2, ldb, 1};
    const int64_t na = gemm_fp4_scale_bytes(M, K, format), nb = gemm_fp4_scale_bytes(N, K, format);
    const Mat sa{sfa, 1, na, na, 1}, sb{sfb, 1, nb, nb, 1}, ga{scale_a, 1, 1, 1, 4}, gb{scale_b, 1, 1, 1, 4};
    for (const Mat *m : {&ma, &mb})
        if ((s = check_mat(*m)) != GEMM_OK) return s;
    if (!sfa || !sfb) return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(sfa) || !aligned16(sfb) || ((reinterpret_cast<uintptr_t>(scale_a) | reinterpret_cast<uintptr_t>(scale_b)) & 3u))
        return GEMM_ERR_MISALIGNED;
    // scale tiles are addressed by a 32-bit coordinate
    if (na / b200::kScaleTile > kMaxDim || nb / b200::kScaleTile > kMaxDim) return GEMM_ERR_TOO_LARGE;
    for (const Mat *m : {&ma, &mb, &sa, &sb, &ga, &gb})
        if (overlap(mc, *m)) return GEMM_ERR_ALIAS;
    DeviceStatus *status;
    if ((s = b200::host::device_with_status(dev, sm_count, status, stream)) != GEMM_OK) return s;
    Fp4Call c{ma, mb, sfa, sfb, format, {}};
    c.args.ga = scale_a;
    c.args.gb = scale_b;
    c.args.c = C;
    c.args.ldc = ldc;
    c.args.M = static_cast<int>(M);
    c.args.N = static_cast<int>(N);
    c.args.K = static_cast<int>(K);
    c.args.tiles_k = static_cast<int>(scale_tiles_k(K, format));
    c.args.f32 = c_type == GEMM_OUT_F32;
    c.args.status = status;
    c.args.timeout_ns = b200::host::watchdog_ns(K);
    return format == GEMM_FP4_NV ? dispatch_fp4<true>(dev, sm_count, c, stream)
                                 : dispatch_fp4<false>(dev, sm_count, c, stream);
}

gemm_status_t gemm_call(gemm_call_t entry, const void *words) {
    static const int kWords[4] = {15, 16, 12, 16};
    if (!words || static_cast<int>(entry) < 0 || static_cast<int>(entry) > GEMM_CALL_FP4) return GEMM_ERR_INVALID_VALUE;
    int64_t w[16];
    std::memcpy(w, words, 8 * static_cast<size_t>(kWords[entry]));
    bool fits = true;
    const auto ptr = [&](int i) { return reinterpret_cast<void *>(static_cast<uintptr_t>(w[i])); };
    const auto code = [&](int i) {
        fits = fits && w[i] == static_cast<int>(w[i]);
        return static_cast<int>(w[i]);
    };
    const auto type = [&](int i) { return static_cast<gemm_out_t>(code(i)); };
    const auto layout = [&](int i) { return static_cast<gemm_layout_t>(code(i)); };
    const auto format = [&](int i) { return static_cast<gemm_fp4_t>(code(i)); };
    const auto stream = [&](int i) { return static_cast<cudaStream_t>(ptr(i)); };
    switch (entry) {
        case GEMM_CALL_BF16_GROUPED: {
            const gemm_out_t c_type = type(12);
            const gemm_layout_t b_layout = layout(13);
            if (!fits) return GEMM_ERR_INVALID_VALUE;
            return gemm_bf16_grouped(ptr(0), ptr(1), static_cast<const int32_t *>(ptr(2)), ptr(3), w[4], w[5], w[6], w[7],
                                     w[8], w[9], w[10], w[11], c_type, b_layout, stream(14));
        }
        case GEMM_CALL_BF16_GROUPED_WGRAD: {
            const gemm_out_t db_type = type(12);
            const gemm_layout_t db_layout = layout(13);
            if (!fits) return GEMM_ERR_INVALID_VALUE;
            float beta;
            std::memcpy(&beta, &w[14], 4);
            return gemm_bf16_grouped_wgrad(ptr(0), ptr(1), static_cast<const int32_t *>(ptr(2)), ptr(3), w[4], w[5], w[6],
                                           w[7], w[8], w[9], w[10], w[11], db_type, db_layout, beta, stream(15));
        }
        case GEMM_CALL_FP4_QUANTIZE: {
            const gemm_fp4_t form = format(8);
            const gemm_out_t x_type = type(9);
            const gemm_layout_t x_layout = layout(10);
            if (!fits) return GEMM_ERR_INVALID_VALUE;
            return gemm_fp4_quantize(ptr(0), static_cast<const float *>(ptr(1)), static_cast<uint8_t *>(ptr(2)),
                                     static_cast<uint8_t *>(ptr(3)), w[4], w[5], w[6], w[7], form, x_type, x_layout,
                                     stream(11));
        }
        default: {
            const gemm_fp4_t form = format(13);
            const gemm_out_t c_type = type(14);
            if (!fits) return GEMM_ERR_INVALID_VALUE;
            return gemm_fp4(static_cast<const uint8_t *>(ptr(0)), static_cast<const uint8_t *>(ptr(1)),
                            static_cast<const float *>(ptr(2)), static_cast<const uint8_t *>(ptr(3)),
                            static_cast<const uint8_t *>(ptr(4)), static_cast<const float *>(ptr(5)), ptr(6), w[7], w[8],
                            w[9], w[10], w[11], w[12], form, c_type, stream(15));
        }
    }
}

}  // extern "C"
