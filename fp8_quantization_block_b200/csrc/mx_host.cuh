// mx_host.cuh -- host side shared by the translation units of libmx.so: the
// settings of mx_debug_set, sizes of the formats, tensor maps, launch
// attributes and argument checks.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>
#include <mutex>
#include <set>
#include <utility>

#include "gemm_sm100.cuh"
#include "mx.h"
#include "mx_common.cuh"

namespace mx {

inline std::atomic<uint64_t> g_wait_limit_ns{1000000000ull};
inline std::atomic<int> g_skip_producer{0};
inline std::atomic<int> g_pair_enabled{1};
inline std::atomic<int> g_pdl_enabled{1};
inline std::atomic<int> g_max_gemm_ctas{0};  // 0: one CTA (or CTA pair) per SM pair of the device
inline std::atomic<int> g_fused_mode{MX_FUSED_PIPELINED};  // how mx_gemm_fused_act runs (MX_DEBUG_FUSED_MODE)
inline std::atomic<int> g_ksplit_mode{0};  // MX_DEBUG_K_SPLIT: 0 auto, 1 never, 2 whenever possible

// Launch attributes shared by the kernels that may overlap the previous kernel
// in the stream (they call griddep_wait() before reading any input).
inline int pdl_attr(cudaLaunchAttribute *a) {
    if (!g_pdl_enabled.load()) return 0;
    a->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a->val.programmaticStreamSerializationAllowed = 1;
    return 1;
}

inline bool valid_fmt(int fmt) { return fmt >= 0 && fmt <= 5; }   // the microscaling formats
inline bool b128_fmt(int fmt) { return fmt == MX_FP8_B128 || fmt == MX_FP8_B128X128; }
inline bool valid_fmt_any(int fmt) { return valid_fmt(fmt) || b128_fmt(fmt); }
inline int fmt_block(int fmt) {
    return b128_fmt(fmt) ? 128 : (fmt == MX_NVFP4 || fmt == MX_MXFP4_MBS) ? 16 : 32;
}
inline int fmt_bits(int fmt) {
    return (fmt == MX_MXFP4 || fmt == MX_NVFP4 || fmt == MX_MXFP4_MBS) ? 4 : (fmt == MX_MXFP6_E3M2 ? 6 : 8);
}
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Blocking granularity a format needs along K (MXFP4-MBS: its 128-element macro blocks).
inline int fmt_k_multiple(int fmt) { return fmt == MX_MXFP4_MBS ? 128 : fmt_block(fmt); }
// Scale tiles, and for MXFP4-MBS the macro mantissas after them ([rows][cols/128], padded to 16).
inline size_t tile_bytes(int fmt, int64_t rows, int64_t cols) {
    return (size_t)(cdiv(rows, 128) * 128 * cdiv(cols / fmt_block(fmt), 4) * 4);
}
// FP8_B128: FP32 scales K block by K block, each block's rows padded to a
// multiple of four so that every block starts on 16 bytes.
inline int64_t b128_pitch(int64_t rows) { return cdiv(rows, 4) * 4; }
inline size_t scales_bytes(int fmt, int64_t rows, int64_t cols) {
    if (fmt == MX_FP8_B128) return (size_t)(4 * b128_pitch(rows) * (cols / 128));
    if (fmt == MX_FP8_B128X128) return (size_t)(cdiv(4 * cdiv(rows, 128) * (cols / 128), 16) * 16);
    size_t t = tile_bytes(fmt, rows, cols);
    if (fmt == MX_MXFP4_MBS) t += (size_t)(cdiv(rows * (cols / 128), 16) * 16);
    return t;
}
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline mx_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MX_OK : MX_ERR_CUDA; }

inline mx_status last_launch() {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        fprintf(stderr, "libmx: launch failed: %s\n", cudaGetErrorString(e));
        return MX_ERR_CUDA;
    }
    return MX_OK;
}

// --- cuTensorMapEncodeTiled through the runtime's driver entry point ---------
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 2D uint8 tensor [rows x row_bytes] (row pitch = row_bytes), box 128 bytes x box_rows, 128-byte swizzle.
inline bool make_tmap_u8(CUtensorMap *m, const void *base, int64_t rows, int64_t row_bytes, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Codes of a kind::mxf8f6f4 operand as a 2D tensor of K elements per row, box
// 128 elements x box_rows, 128-byte swizzle.  Every type lands in shared memory
// as 128 bytes per row: FP8 bytes as they are; FP6 (16 codes in 12 bytes) and
// FP4 (16 codes in 8 bytes) unpacked by the copy to one 16-byte group per 16
// codes, the layout the MMA reads for these types.  The sub-byte types need a
// 32-byte aligned base, row pitches that are multiples of 32 bytes and K a
// multiple of 128 (the caller checks).
inline bool make_tmap_codes_f8f6f4(CUtensorMap *m, int fmt, const void *base, int64_t rows, int64_t K, int box_rows) {
    if (fmt_bits(fmt) == 8) return make_tmap_u8(m, base, rows, K, box_rows);
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const CUtensorMapDataType dt =
        fmt_bits(fmt) == 6 ? CU_TENSOR_MAP_DATA_TYPE_16U6_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(K * fmt_bits(fmt) / 8)};
    cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = fn(m, dt, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) fprintf(stderr, "libmx: tensor map for format %d codes failed (%d)\n", fmt, (int)r);
    return r == CUDA_SUCCESS;
}

// Formats that kind::mxf8f6f4 multiplies (E8M0 scales on 32-element blocks),
// and their element-type codes in its instruction descriptor.
inline bool f8f6f4_fmt(int fmt) {
    return fmt == MX_MXFP8_E4M3 || fmt == MX_MXFP8_E5M2 || fmt == MX_MXFP4 || fmt == MX_MXFP6_E3M2;
}
inline uint32_t f8f6f4_type(int fmt) {
    switch (fmt) {
    case MX_MXFP8_E4M3: return kTypeE4M3;
    case MX_MXFP8_E5M2: return kTypeE5M2;
    case MX_MXFP6_E3M2: return kTypeE3M2;
    default: return kTypeE2M1;
    }
}
// Can A and B be multiplied, and on which kernel: the format's own (same
// format, 0..3) or the run-time-typed kind::mxf8f6f4 one.
inline bool gemm_pair_ok(int fa, int fb) {
    return (fa == fb && (fa <= MX_NVFP4 || fa == MX_MXFP4_MBS)) || (f8f6f4_fmt(fa) && f8f6f4_fmt(fb)) ||
           (fa == MX_FP8_B128 && fb == MX_FP8_B128X128);
}
inline bool gemm_runtime_types(int fa, int fb) { return !(fa == fb && (fa <= MX_NVFP4 || fa == MX_MXFP4_MBS)); }
inline bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// SM count of the current device, read once per device.
inline int num_sms() {
    constexpr int kMaxDev = 64;
    static std::atomic<int> cache[kMaxDev];
    int dev = 0;
    cudaGetDevice(&dev);
    const bool cached = dev >= 0 && dev < kMaxDev;
    int n = cached ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        if (cached) cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

inline mx_status check_tensor(const mx_tensor *t, bool need_codes) {
    if (!t || !valid_fmt_any(t->fmt) || t->rows < 0 || t->cols < 0) return MX_ERR_INVALID_ARG;
    if (t->cols % fmt_k_multiple(t->fmt) != 0) return MX_ERR_UNSUPPORTED_SHAPE;
    if (t->rows > 0 && t->cols > 0) {
        if (need_codes && (!t->codes || !t->scales)) return MX_ERR_INVALID_ARG;
        if (!aligned16(t->codes) || !aligned16(t->scales)) return MX_ERR_MISALIGNED;
        if (t->fmt == MX_NVFP4 && !t->gscale) return MX_ERR_INVALID_ARG;
    }
    return MX_OK;
}

// bf16 [rows x cols] output (row pitch ld elements), box 32 x 32, no swizzle.
inline bool make_tmap_c(CUtensorMap *m, void *base, int64_t rows, int64_t cols, int64_t ld) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(ld * 2)};
    cuuint32_t box[2] = {32u, 32u};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Scale tiles as a 3D tensor of 8-byte words: [bands][sf_tiles_k][64] (one
// 512-byte tile = 64 words), box = box_chunks tiles of box_bands bands.  Reads
// past either end (a ragged K or N) return zeros.
inline bool make_tmap_sf(CUtensorMap *m, const uint8_t *scales, int64_t bands, int64_t sf_tiles_k, int box_chunks,
                  int box_bands) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {64u, (cuuint64_t)sf_tiles_k, (cuuint64_t)bands};
    cuuint64_t strides[2] = {512u, (cuuint64_t)(sf_tiles_k * 512)};
    cuuint32_t box[3] = {64u, (cuuint32_t)box_chunks, (cuuint32_t)box_bands};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 3, const_cast<uint8_t *>(scales), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Raise the dynamic shared memory limit of kernel fn to `bytes` on the current
// device, once per (kernel, device): the attribute belongs to the device's
// context, so a process that drives several GPUs sets it on each.
inline cudaError_t smem_limit_once(const void *fn, int bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    static std::mutex mu;
    static std::set<std::pair<const void *, int>> done;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count({fn, dev}) != 0) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.insert({fn, dev});
    return e;
}

// --- mx_experts.cu -------------------------------------------------------
mx_status quantize_b128(int fmt, const uint16_t *src, int64_t M, int64_t K, int64_t ld, const mx_tensor *dst,
                        cudaStream_t st);
mx_status dequantize_b128(const mx_tensor *src, uint16_t *dst, int64_t ld, cudaStream_t st);
mx_status gemm_b128(const mx_tensor *A, const mx_tensor *B, uint16_t *C, int64_t ldc, int epilogue, cudaStream_t st);
mx_status experts_error_word(uint32_t w[4]);

}  // namespace mx
