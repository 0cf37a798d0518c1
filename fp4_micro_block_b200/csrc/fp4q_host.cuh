// fp4q_host.cuh -- host side shared by the library's translation units: device
// information, TMA descriptor encoding, argument checks and kernel launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <utility>

#include "../../include/fp4q.h"

#define FP4Q_API extern "C" __attribute__((visibility("default")))

namespace fp4q {

constexpr int kMaxGrid = 4096;  // partial maxima fit FP4Q_WORKSPACE_BYTES
static_assert(kMaxGrid * sizeof(float) <= FP4Q_WORKSPACE_BYTES, "workspace too small");

// ---------------------------------------------------------------- device info
constexpr int kMaxDevices = 64;
inline std::atomic<int> g_sm_count[kMaxDevices];

inline fp4q_status sm_count(int* out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FP4Q_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return FP4Q_ERR_UNSUPPORTED;
    int n = g_sm_count[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return FP4Q_ERR_CUDA;
        g_sm_count[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return FP4Q_OK;
}

// ---------------------------------------------------------------- TMA descriptors
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline std::atomic<EncodeTiledFn> g_encode{nullptr};

inline fp4q_status encode_fn(EncodeTiledFn* out) {
    EncodeTiledFn fn = g_encode.load(std::memory_order_acquire);
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !p)
            return FP4Q_ERR_CUDA;
        fn = reinterpret_cast<EncodeTiledFn>(p);
        g_encode.store(fn, std::memory_order_release);
    }
    *out = fn;
    return FP4Q_OK;
}

// bf16 [M, K] with row stride ldx elements; boxes of 64 columns x box_rows rows
// (8: the G2 warp-tile halves; 128: the tensor-core tile halves), 128-byte
// swizzle, zero fill outside the matrix.
inline fp4q_status make_x_map(CUtensorMap* map, const void* x, int64_t M, int64_t K, int64_t ldx,
                       uint32_t box_rows = 8) {
    EncodeTiledFn enc;
    fp4q_status st = encode_fn(&enc);
    if (st != FP4Q_OK) return st;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)M};
    cuuint64_t strides[1] = {(cuuint64_t)ldx * 2};
    cuuint32_t box[2] = {64u, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(x), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP4Q_OK : FP4Q_ERR_CUDA;
}

// uint8 [rows, row_bytes] (packed E2M1 codes), boxes of 128 bytes x box_rows
// rows with the 128-byte swizzle, zero fill outside the matrix.
inline fp4q_status make_codes_map(CUtensorMap* map, const void* codes, int64_t rows, int64_t row_bytes,
                           uint32_t box_rows) {
    EncodeTiledFn enc;
    fp4q_status st = encode_fn(&enc);
    if (st != FP4Q_OK) return st;
    cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    cuuint32_t box[2] = {128u, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box,
                     estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP4Q_OK : FP4Q_ERR_CUDA;
}

// Row-major [rows, cols] of 1-byte or 4-byte elements (row stride row_bytes, a
// multiple of 16), boxes of box_cols x box_rows, no swizzle, zero fill outside.
inline fp4q_status make_plain_map(CUtensorMap* map, CUtensorMapDataType dt, const void* base, int64_t rows, int64_t cols,
                           int64_t row_bytes, uint32_t box_cols, uint32_t box_rows) {
    EncodeTiledFn enc;
    fp4q_status st = encode_fn(&enc);
    if (st != FP4Q_OK) return st;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP4Q_OK : FP4Q_ERR_CUDA;
}

// Packed codes [rows, row_bytes] written by TMA stores of box_bytes x 128 rows
// (64-byte boxes with the 64-byte swizzle, 128-byte boxes with the 128-byte
// one); rows past `rows` are not written.
inline fp4q_status make_codes_store_map(CUtensorMap* map, void* codes, int64_t rows, int64_t row_bytes,
                                 uint32_t box_bytes) {
    EncodeTiledFn enc;
    fp4q_status st = encode_fn(&enc);
    if (st != FP4Q_OK) return st;
    cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    cuuint32_t box[2] = {box_bytes, 128u};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE,
                     box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP4Q_OK : FP4Q_ERR_CUDA;
}

// bf16 [rows, cols] output (row stride cols * 2 bytes, a multiple of 16) stored
// by the TMA in boxes of 32 columns x 128 rows with the 64-byte swizzle; rows
// past `rows` are not written.
inline fp4q_status make_bf16_store_map(CUtensorMap* map, void* base, int64_t rows, int64_t cols) {
    EncodeTiledFn enc;
    fp4q_status st = encode_fn(&enc);
    if (st != FP4Q_OK) return st;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(cols * 2)};
    cuuint32_t box[2] = {32u, 128u};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP4Q_OK : FP4Q_ERR_CUDA;
}

// ---------------------------------------------------------------- validation
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxDim = (int64_t)1 << 31;

inline fp4q_status check_x(const void* x, int64_t M, int64_t K, int64_t ldx) {
    if (M < 0 || K <= 0 || ldx < K) return FP4Q_ERR_INVALID_ARG;
    if (M >= kMaxDim || K >= kMaxDim || ldx >= kMaxDim) return FP4Q_ERR_UNSUPPORTED;
    if (K < 64) return FP4Q_ERR_UNSUPPORTED;
    if (M > 0 && !x) return FP4Q_ERR_INVALID_ARG;
    if (ldx % 8 != 0 || !aligned(x, 16)) return FP4Q_ERR_ALIGNMENT;
    return FP4Q_OK;
}

inline fp4q_status check_out(const uint8_t* codes, const uint8_t* scales) {
    if (!codes || !scales) return FP4Q_ERR_INVALID_ARG;
    if (!aligned(codes, 16) || !aligned(scales, 4)) return FP4Q_ERR_ALIGNMENT;
    return FP4Q_OK;
}

// Launches kern on stream s with programmatic stream serialization, so the
// kernel's prologue may overlap the end of the previous kernel in the stream
// (each kernel waits in pdl_wait() before it touches global memory).
template <typename... KArgs, typename... Args>
inline fp4q_status launch(void (*kern)(KArgs...), int grid, int threads, int smem, cudaStream_t s, Args&&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) == cudaSuccess ? FP4Q_OK : FP4Q_ERR_CUDA;
}

inline fp4q_status launch_status() {
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FP4Q_OK : FP4Q_ERR_CUDA;
}

// Raises a kernel's dynamic shared-memory limit once per device (the attribute
// is per function and device; setting it again is harmless but costs host time).
template <typename Kern>
inline fp4q_status ensure_smem(Kern kern, int bytes, std::atomic<uint64_t>& done) {
    if (bytes <= 48 * 1024) return FP4Q_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FP4Q_ERR_CUDA;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return FP4Q_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return FP4Q_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_acq_rel);
    return FP4Q_OK;
}

}  // namespace fp4q
