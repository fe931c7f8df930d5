// Host helpers that every entry point's source file shares: the device check,
// the record behind gemm_last_cuda_error, overlap and alignment tests.
// Defined in b200gemm.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <atomic>
#include <cstdint>

#include "b200gemm.h"

namespace b200 {

struct DeviceStatus;

namespace host {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxDim = 0x7FFFFFFF;

// Records the error for gemm_last_cuda_error.
gemm_status_t cuda_fail(cudaError_t e);

// The current device, checked to be compute capability 10.0, and its number
// of SMs.  Allocates nothing; the first call on a device may not be captured
// (GEMM_ERR_CAPTURE).
gemm_status_t device(int &dev, int &sm_count, cudaStream_t stream);

// The same, with the device's watchdog status block (allocated on the first
// call on the device that needs it).
gemm_status_t device_with_status(int &dev, int &sm_count, DeviceStatus *&status, cudaStream_t stream);

// How long a wait inside a kernel with a reduction of length K may take.
uint64_t watchdog_ns(int64_t K);

// A tensor map of `rank` (2 or 3) dimensions, innermost first, without
// interleaving, zeros outside.  strides: bytes, of the outer dimensions.
gemm_status_t encode_map(CUtensorMap *map, CUtensorMapDataType dtype, const void *ptr, int rank, const int64_t *dims,
                         const int64_t *strides, const uint32_t *box, CUtensorMapSwizzle swizzle);

// True while `stream` is being captured into a CUDA graph.
bool capturing(cudaStream_t stream);

// Whether the byte ranges of two row-major matrices (rows x cols of `esize`
// bytes with leading dimension ld) overlap.
bool overlaps(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t esize, const void *q, int64_t qrows,
              int64_t qcols, int64_t qld, int64_t qesize);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether a pitch of ld >= 0 elements is a multiple of 16 bytes.  The product
// ld * esize may not be formed before extent_ok has bounded ld: it wraps for
// pitches near 2^62 elements.
inline bool pitch16(int64_t ld, int64_t esize) { return (ld % 16) * esize % 16 == 0; }

// Whether a matrix of `rows` rows with pitch ld keeps within the limits that
// every offset is computed under: a pitch below 2^40 bytes (the tensor maps'
// limit), and at most 2^62 bytes from the first row to the last (far above any
// address space), so that no byte offset wraps, here or in a kernel.
inline bool extent_ok(int64_t rows, int64_t ld, int64_t esize) {
    if (ld >= (int64_t(1) << 40) / esize) return false;
    return rows <= 1 || ld == 0 || rows <= (int64_t(1) << 62) / (ld * esize);
}

// One-time set-up of a kernel on a device: loads it (lazy loading may not
// happen inside a stream capture) and raises its dynamic shared memory limit.
// `Kernel` gives each kernel flags of its own, one bit per device.
template <auto Kernel>
gemm_status_t prepare(int dev, int smem_bytes, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    const uint64_t bit = uint64_t(1) << dev;
    if (ready.load(std::memory_order_acquire) & bit) return GEMM_OK;
    if (capturing(stream)) return GEMM_ERR_CAPTURE;
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, Kernel);
    if (e == cudaSuccess && smem_bytes > 48 * 1024)
        e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
    if (e != cudaSuccess) return cuda_fail(e);
    ready.fetch_or(bit, std::memory_order_release);
    return GEMM_OK;
}

}  // namespace host
}  // namespace b200
