// quantize_b128.cuh -- E4M3 codes with one FP32 scale per block of 128 along K,
// and the quantize of rows gathered by expert.
//
//   scale   s = RN_fp32(max|x| / 448) over the block: 1 x 128 elements
//           (MX_FP8_B128, activations) or 128 x 128 (MX_FP8_B128X128, weights);
//   element q = RNE_e4m3(x / s) of the exact quotient, saturating at 448; a
//           block of zeros has s = 0 and the signed zeros of x.
//
// A quotient of a bf16 value and an FP32 scale often lies next to the middle
// of two codes (x and max|x| are short numbers, and s is max|x| / 448 but for
// one rounding), so rounding the quotient to FP32 first would change codes.
// As for NVFP4, two products with 1/s rounded down and up bracket it, both
// cast; where their codes differ the sign of |x| - s * middle, exact in one
// fma, decides.
//
// Bound by HBM: 2 bytes read and 1 written per element (+ 4/128 per row block).
#pragma once

#include "groups.cuh"
#include "quantize.cuh"

namespace mx {

// Scale of a block and the bracket of its reciprocal.  Below 2^-60 the values
// and the scale are multiplied by 2^64 first (both exact), so that neither the
// reciprocal nor the products leave the normal range.
struct B128Scale {
    float s;            // the scale as stored
    float ss;           // s times sc
    float r_lo, r_hi;
    float sc;
};
MX_DEVICE_INLINE B128Scale b128_scale(uint32_t amax_bits) {
    B128Scale b;
    const float amax = __uint_as_float(amax_bits << 16);
    b.s = __fdiv_rn(amax, 448.0f);
    b.sc = amax < 0x1p-60f ? 0x1p64f : 1.0f;
    b.ss = b.s * b.sc;
    b.r_lo = amax_bits != 0u ? __frcp_rd(b.ss) : 0.0f;
    b.r_hi = amax_bits != 0u ? __frcp_ru(b.ss) : 0.0f;
    return b;
}

// Settle the bytes of a word of four codes whose bracket straddles a middle:
// diff is nonzero in those bytes; w0, w1 hold the four bf16 inputs.
MX_DEVICE_INLINE uint32_t b128_settle(uint32_t code, uint32_t diff, uint32_t w0, uint32_t w1, const B128Scale &b) {
    while (diff != 0u) {
        const int i = (__ffs(diff) - 1) >> 3;
        diff &= ~(0xFFu << (8 * i));
        const uint32_t w = i < 2 ? w0 : w1;
        const float ax = fabsf((i & 1) ? bf16hi(w) : bf16lo(w)) * b.sc;
        const uint32_t c = (code >> (8 * i)) & 0x7Fu;   // the lower code, below 0x7E (448)
        const float mid = 0.5f * ((c ? e4m3_pos_value(c) : 0.0f) + e4m3_pos_value(c + 1u));
        const float d = __fmaf_rn(-b.ss, mid, ax);
        if (d > 0.0f || (d == 0.0f && (c & 1u))) code += 1u << (8 * i);
    }
    return code;
}

// E4M3 codes of 16 bf16 values under one scale.
MX_DEVICE_INLINE uint4 b128_codes16(const uint4 &v0, const uint4 &v1, const B128Scale &b) {
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint64_t P[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) P[i] = pk2(bf16lo(w[i]), bf16hi(w[i]));
    if (b.sc != 1.0f) {
        const uint64_t SC = pk2(b.sc, b.sc);
#pragma unroll
        for (int i = 0; i < 8; ++i) P[i] = mul2(P[i], SC);
    }
    float lo[16], hi[16];
    bracket16(P, b.r_lo, b.r_hi, lo, hi);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] = cvt4_fp8<FMT_E4M3>(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
        const uint32_t h = cvt4_fp8<FMT_E4M3>(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
        const uint32_t d = (c[i] ^ h) & 0x7F7F7F7Fu;
        if (d != 0u) c[i] = b128_settle(c[i], d, w[2 * i], w[2 * i + 1], b);
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
}

struct B128QuantParams {
    const uint16_t *src;
    int64_t ld;
    int64_t src_rows;            // rows of src (a gather's indexes are checked against it)
    const int32_t *row_index;    // nullable: source row of each output row
    const int32_t *offsets;      // nullable: rows from offsets[groups] on are left as they are
    int groups;
    int64_t M, K;
    uint8_t *codes;
    float *scales;
    int64_t pitch;               // 1 x 128: floats per K block; 128 x 128: floats per row of scales
};

// One CTA per 128 x 128 tile, as quantize_kernel: 8 lanes per row, 16 elements
// per lane and pass, all loads issued before the first use.
template <bool TILE, bool GROUPED>
__global__ void __launch_bounds__(kQThreads) quantize_b128_kernel(B128QuantParams p) {
    constexpr int kPasses = kQTileRows / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = (int64_t)blockIdx.y * kQTileRows;
    const int64_t kb = blockIdx.x;
    const int64_t col = kb * kQTileCols + (lane & 7) * 16;
    griddep_wait();
    griddep_launch_dependents();
    int64_t live = p.M;
    if (GROUPED) live = min((int64_t)max(p.offsets[p.groups], 0), p.M);
    uint4 v[kPasses][2];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t row = row0 + i * 32 + warp * 4 + (lane >> 3);
        v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (row < live) {
            int64_t from = row;
            if (GROUPED && p.row_index != nullptr) from = p.row_index[row];
            if (!GROUPED || (from >= 0 && from < p.src_rows)) {
                const uint16_t *s = p.src + from * p.ld + col;
                v[i][0] = ldg_stream(s);
                v[i][1] = ldg_stream(s + 8);
            }
        }
    }
    if (TILE) {
        __shared__ uint32_t red[kQThreads / 32];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) m = max(m, absmax16(v[i][0], v[i][1]));
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) red[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kQThreads / 32; ++w) m = max(m, red[w]);
        const B128Scale b = b128_scale(m);
        if (threadIdx.x == 0) p.scales[(int64_t)blockIdx.y * p.pitch + kb] = b.s;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int64_t row = row0 + i * 32 + warp * 4 + (lane >> 3);
            if (row < live) *reinterpret_cast<uint4 *>(p.codes + row * p.K + col) = b128_codes16(v[i][0], v[i][1], b);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int64_t row = row0 + i * 32 + warp * 4 + (lane >> 3);
            uint32_t m = absmax16(v[i][0], v[i][1]);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
            const B128Scale b = b128_scale(m);
            if (row < live) *reinterpret_cast<uint4 *>(p.codes + row * p.K + col) = b128_codes16(v[i][0], v[i][1], b);
            // the scales' padding up to the pitch is 0 (a grouped call leaves rows past the last group alone)
            if ((lane & 7) == 0 && row < (GROUPED ? live : p.pitch)) p.scales[kb * p.pitch + row] = b.s;
        }
    }
}

// bf16(s * q), the product exact before its one rounding (FP64 holds it).
__global__ void __launch_bounds__(256) dequantize_b128_kernel(const uint8_t *__restrict__ codes,
                                                              const float *__restrict__ scales, int64_t rows,
                                                              int64_t cols, int64_t row_div, int64_t row_step,
                                                              int64_t kb_step, uint16_t *__restrict__ dst, int64_t ld) {
    const int64_t segs = cols / 8;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    griddep_wait();
    if (i >= rows * segs) return;
    const int64_t r = i / segs, c = (i % segs) * 8;
    const double s = scales[(r / row_div) * row_step + (c / 128) * kb_step];
    const uint2 w = *reinterpret_cast<const uint2 *>(codes + r * cols + c);
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t code = ((j < 2 ? w.x : w.y) >> (16 * (j & 1) + 8 * e)) & 0xFFu;
            const uint32_t mag = code & 0x7Fu;
            const double q = mag == 0x7Fu ? (double)__uint_as_float(0x7FC00000u)
                                          : (mag ? (double)e4m3_pos_value(mag) : 0.0);
            const __nv_bfloat16 b = __double2bfloat16(s * q);
            h |= (uint32_t)(__bfloat16_as_ushort(b) ^ ((code & 0x80u) << 8)) << (16 * e);
        }
        out[j] = h;
    }
    *reinterpret_cast<uint4 *>(dst + r * ld + c) = make_uint4(out[0], out[1], out[2], out[3]);
}

// Quantize of rows grouped by expert into a format whose scales come in
// 128-row tiles: each group begins a 128-row band of the scale buffer, so the
// grouped GEMM's 128-row tiles read whole bands.  CTA (tile, band) finds its
// group by a warp's walk and then quantizes 128 x 128 elements exactly as
// quantize_kernel; bands past the last group's get zero scales.
struct GroupedQuantParams {
    const uint16_t *src;
    int64_t ld;
    int64_t src_rows;
    const int32_t *row_index;    // nullable
    Groups groups;
    int64_t K;
    uint8_t *codes;
    uint8_t *scales;
    int64_t sf_tiles_k;
    const float *gscale;         // NVFP4: g
    float *gscale_out;           // NVFP4, nullable: receives g
};

template <int FMT>
__global__ void __launch_bounds__(kQThreads, quantize_min_blocks<FMT>()) quantize_grouped_kernel(GroupedQuantParams p) {
    constexpr int kPasses = kQTileRows / 32;
    __shared__ __align__(16) uint8_t sf_tile[quantize_sf_bytes<FMT>()];
    __shared__ NvTables nvt;
    __shared__ int info[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col0 = (int64_t)blockIdx.x * kQTileCols;
    const int cl = (lane & 7) * 16;
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 0) {
        GroupWalk walk(p.groups, 7, lane);
        GroupBlock b;
        int r0 = 0, r1 = 0;
        if (walk.find((int)blockIdx.y, b)) {
            r0 = b.start + ((int)blockIdx.y - b.first) * kQTileRows;
            r1 = min(b.end, r0 + kQTileRows);
        }
        if (lane == 0) {
            info[0] = r0;
            info[1] = r1;
        }
    }
    NvScale ns{1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    if (FMT == FMT_NVFP4) {
        const float g = *p.gscale;
        if (p.gscale_out != nullptr && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.gscale_out = g;
        ns = nv_scale_setup(g);
        if (threadIdx.x < 128) nv_tables_fill(&nvt, threadIdx.x);
    }
    __syncthreads();
    const int64_t row0 = info[0], row1 = info[1];
    uint4 v[kPasses][2];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t row = row0 + i * 32 + warp * 4 + (lane >> 3);
        v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (row < row1 && col0 + cl < p.K) {
            const int64_t from = p.row_index != nullptr ? p.row_index[row] : row;
            if (from >= 0 && from < p.src_rows) {
                const uint16_t *s = p.src + from * p.ld + col0 + cl;
                v[i][0] = ldg_stream(s);
                v[i][1] = ldg_stream(s + 8);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int rl = i * 32 + warp * 4 + (lane >> 3);
        quantize_seg16<FMT, RULE_OCP>(v[i][0], v[i][1], row0 + rl, row1, col0 + cl, p.K, col0, rl, cl, lane, ns, &nvt,
                                      p.codes, sf_tile);
    }
    __syncthreads();
    store_sf_chunks<FMT>(sf_tile, p.scales, blockIdx.y, blockIdx.x, p.sf_tiles_k, threadIdx.x);
}

}  // namespace mx
