// gemm_b128_sm100.cuh -- GEMM of E4M3 matrices with one FP32 scale per block
// of 128 along K, on the sm_100a tensor cores; plain or grouped by expert.
//
//   C[i][j] = sum_b sA[i][b] sB[j / 128][b] P_b[i][j],
//   P_b[i][j] = sum over the 128 elements k of block b of qA[i][k] qB[j][k],
//
// qA, qB E4M3, A with a scale per row and block, B with one per 128 x 128.  The
// scales are arbitrary FP32 numbers, which the tensor core's own block scales
// (powers of two) cannot carry, so P_b is formed in TMEM by kind::f8f6f4 and
// scaled on the way out: one thread owns one row, so sA sB is one number per
// thread and 128-column block, and a packed fma folds two columns of P_b into
// the running sums, which stay in registers (FP32) for the whole tile.
//
// Persistent kernel, 12 warps:
//   warp 0       TMA producer of A and B (128 bytes of K = one block per
//                stage, 128-byte swizzle) into a ring that runs on across tiles;
//   warp 1       TMEM owner and MMA issuer: 4 MMAs of K = 32 per stage into one
//                of the partial buffers (2 of 256 columns, or 4 of 128), which
//                then holds that block's P_b alone;
//   warps 4-11   two per TMEM lane quadrant: drain a partial buffer (half of
//                its columns each) while the next block's MMAs run, then
//                [GELU], bf16 and store after the last block.
// Registers move from warps 0-3 to the drain warps (setmaxnreg), whose sums
// take 128 of them each for 256-column tiles.
//
// Tile sizes are run-time numbers: bm rows (32, 64, 128, or 256 on a CTA pair)
// and bn columns (a multiple of 32 up to 256), so that few-row products, which
// are bound by the weight stream, spread over all SMs.  PAIR: two CTAs share a
// 256 x bn tile with cta_group::2 MMAs, each loading its own 128 rows of A and
// half of B: per SM half the B traffic for the same MMAs.
#pragma once

#include "gemm_sm100.cuh"
#include "groups.cuh"

namespace mx {

constexpr int kB128Threads = 384;
constexpr int kB128DrainWarps = 8;
constexpr int kB128MaxStages = 16;
constexpr int kB128StagingBytes = kB128DrainWarps * 2 * kEpiChunkBytes;   // two 32 x 32 bf16 buffers per drain warp
// registers per thread: the sum over the three warpgroups is what the block
// is launched with (384 threads at 168)
constexpr int kB128DrainRegs = 216, kB128OtherRegs = 72;
static_assert(2 * kB128DrainRegs + kB128OtherRegs <= 3 * 168, "register split");

struct B128GemmParams {
    const float *sa;       // [K / 128][sa_pitch], by row of A
    const float *sb;       // [groups][sb_step]: [ceil(N / 128)][K / 128]
    uint16_t *C;
    int64_t ldc;
    int64_t sa_pitch;
    int64_t sb_step;       // floats per group
    int M, N;              // rows of A; columns of C (rows of B per group)
    int num_kb;            // K / 128
    int bm_shift;          // log2 of the tile's rows (5 .. 8)
    int bn;
    int m_blocks, n_blocks;
    int stages;
    int a_bytes, b_bytes;  // per stage and CTA
    int epilogue;          // 0 none, 1 GELU
    int use_tma_store;     // C 16-byte aligned, ldc % 8 == 0
    int skip_producer;
    uint64_t wait_limit_ns;
    Groups groups;         // GROUPED
};

// Instruction descriptor of kind::f8f6f4: FP32 accumulator, E4M3 x E4M3, both K-major.
MX_DEVICE_INLINE uint32_t b128_idesc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// A tile's place: rows [row0, row_end) of A and C, columns n0.. of the group.
struct B128Tile {
    int row0, row_end, n0, group;
};

// The tiles in order: within a group (or the whole matrix) rows fastest, so
// that neighbouring CTAs share a slice of B.
template <bool GROUPED>
class B128Tiles {
  public:
    MX_DEVICE_INLINE B128Tiles(const B128GemmParams &p, int lane) : p_(p), walk_(p.groups, p.bm_shift, lane) {}
    MX_DEVICE_INLINE bool at(int t, B128Tile &o) {
        GroupBlock b;
        if (!walk_.find(t / p_.n_blocks, b)) return false;
        const int local = t - b.first * p_.n_blocks;
        const int nb = local / b.blocks;
        o.group = b.group;
        o.n0 = nb * p_.bn;
        o.row0 = b.start + ((local - nb * b.blocks) << p_.bm_shift);
        o.row_end = b.end;
        return true;
    }

  private:
    const B128GemmParams &p_;
    GroupWalk walk_;
};
template <>
class B128Tiles<false> {
  public:
    MX_DEVICE_INLINE B128Tiles(const B128GemmParams &p, int) : p_(p) {}
    MX_DEVICE_INLINE bool at(int t, B128Tile &o) {
        if (t >= p_.m_blocks * p_.n_blocks) return false;
        const int nb = t / p_.m_blocks;
        o.group = 0;
        o.n0 = nb * p_.bn;
        o.row0 = (t - nb * p_.m_blocks) << p_.bm_shift;
        o.row_end = p_.M;
        return true;
    }

  private:
    const B128GemmParams &p_;
};

// One 32-column chunk (rows m0q + lane, columns col ..) of C through this
// warp's staging buffers: a TMA store where all 32 rows are the tile's own (a
// store clips at the matrix's edges, not at a group's), else row by row, each
// row's columns as one coalesced write.
MX_DEVICE_INLINE void b128_store_chunk(const B128GemmParams &p, const CUtensorMap *tmC, const uint32_t (&packed)[16],
                                       int m0q, int row_end, int col, int lane, uint8_t *bufs, uint32_t &nstore) {
    uint8_t *buf = bufs + (nstore & 1u) * kEpiChunkBytes;
    ++nstore;
    if (lane == 0) bulk_wait_group_read<1>();   // this buffer's previous store has read it
    __syncwarp();
    uint4 *dst = reinterpret_cast<uint4 *>(buf + lane * 64);
#pragma unroll
    for (int v = 0; v < 4; ++v)
        dst[v] = make_uint4(packed[4 * v], packed[4 * v + 1], packed[4 * v + 2], packed[4 * v + 3]);
    if (p.use_tma_store && (m0q + 32 <= row_end || row_end == p.M)) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(tmC, col, m0q, buf);
            bulk_commit_group();
        }
    } else {
        __syncwarp();
        const int rows = min(32, row_end - m0q), cols = min(32, p.N - col);
        uint16_t *c = p.C + (int64_t)m0q * p.ldc + col;
        if (p.use_tma_store && cols == 32) {
            // eight rows at a time, 16 bytes per lane
            for (int r = lane >> 2; r < rows; r += 8)
                *reinterpret_cast<uint4 *>(c + (int64_t)r * p.ldc + 8 * (lane & 3)) =
                    *reinterpret_cast<const uint4 *>(buf + r * 64 + 16 * (lane & 3));
        } else {
            for (int r = 0; r < rows; ++r)
                if (lane < cols) c[(int64_t)r * p.ldc + lane] = *reinterpret_cast<const uint16_t *>(buf + r * 64 + 2 * lane);
        }
        __syncwarp();
        if (lane == 0) bulk_commit_group();   // an empty group keeps the buffers' order of groups
    }
}

// CH: 32-column chunks per drain warp (4: tiles of up to 256 columns and two
// partial buffers; 2: up to 128 columns and four partial buffers).
template <bool PAIR, int CH, bool GROUPED>
__global__ void __launch_bounds__(kB128Threads, 1)
    gemm_b128_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const B128GemmParams p) {
    constexpr int kPartialCols = CH * 64;
    constexpr int NP = 512 / kPartialCols;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int S = p.stages;
    uint8_t *smem_a = smem, *smem_b = smem + S * p.a_bytes;
    uint8_t *staging = smem_b + S * p.b_bytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + kB128StagingBytes);   // the pair leader's count both CTAs
    uint64_t *empty = full + kB128MaxStages;
    uint64_t *pfull = empty + kB128MaxStages;   // [NP]
    uint64_t *pempty = pfull + 4;               // [NP], the leader's count both CTAs' drain warps
    uint64_t *mma_done = pempty + 4;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const int worker = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int workers = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < NP; ++i) {
            mbar_init(&pfull[i], 1);
            mbar_init(&pempty[i], (PAIR ? 2 : 1) * kB128DrainWarps);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        if (p.use_tma_store) tma_prefetch_desc(&tmC);
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(tmem_slot, 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, 512);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();   // both CTAs' barriers exist before anyone signals them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();

    if (warp < 4) {
        if (CH == 4) setmaxnreg_dec<kB128OtherRegs>();
        if (warp == 0 && !p.skip_producer) {
            // -------------------------------------------------------- producer
            B128Tiles<GROUPED> tiles(p, lane);
            const uint32_t full_leader0 = PAIR ? mapa_shared(smem_u32(&full[0]), 0) : 0u;
            int used = 0, s = 0;
            uint32_t ph = 0;
            bool stop = false;
            B128Tile t;
            for (int i = worker; !stop && tiles.at(i, t); i += workers) {
                const int a_row = t.row0 + (PAIR ? 128 * (int)rank : 0);
                const int b_row = t.group * p.N + t.n0 + (PAIR ? (p.bn / 2) * (int)rank : 0);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_wait_bounded(&empty[s], ph ^ 1u, p.wait_limit_ns, SITE_GEMM_PRODUCER_EMPTY, abort_flag)) {
                        stop = true;
                        break;
                    }
                    if (lane == 0) {
                        if (PAIR) {
                            const uint32_t bar = full_leader0 + 8u * (uint32_t)s;
                            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * (uint32_t)(p.a_bytes + p.b_bytes));
                            tma_load_2d_pair(smem_a + s * p.a_bytes, &tmA, kb * kStageKBytes, a_row, bar);
                            tma_load_2d_pair(smem_b + s * p.b_bytes, &tmB, kb * kStageKBytes, b_row, bar);
                        } else {
                            mbar_arrive_expect_tx(&full[s], (uint32_t)(p.a_bytes + p.b_bytes));
                            tma_load_2d(smem_a + s * p.a_bytes, &tmA, kb * kStageKBytes, a_row, &full[s]);
                            tma_load_2d(smem_b + s * p.b_bytes, &tmB, kb * kStageKBytes, b_row, &full[s]);
                        }
                    }
                    __syncwarp();
                    ++used;
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // copies in flight land before this CTA (the leader, for both) may leave
            if (rank == 0)
                for (int u = max(0, used - S); u < used; ++u)
                    mbar_wait_bounded(&full[u % S], (uint32_t)((u / S) & 1), p.wait_limit_ns, SITE_GEMM_TAIL, nullptr);
        } else if (warp == 1 && rank == 0) {
            // -------------------------------------------------------- MMA issuer
            const uint64_t desc = smem_desc(0, 16, 1024, 2);
            const uint64_t ad0 = desc | (uint64_t)((smem_u32(smem_a) >> 4) & 0x3FFFu);
            const uint64_t bd0 = desc | (uint64_t)((smem_u32(smem_b) >> 4) & 0x3FFFu);
            const uint32_t idesc = b128_idesc(PAIR ? 256 : 128, p.bn);
            const uint32_t leader = lane == 0 ? 1u : 0u;
            B128Tiles<GROUPED> tiles(p, lane);
            int s = 0, pi = 0;
            uint32_t ph = 0, pph = 0;
            bool stop = false;
            B128Tile t;
            for (int i = worker; !stop && tiles.at(i, t); i += workers) {
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_wait_bounded(&pempty[pi], pph ^ 1u, p.wait_limit_ns, SITE_GEMM_MMA_ACC_EMPTY, abort_flag) ||
                        !mbar_wait_bounded(&full[s], ph, p.wait_limit_ns, SITE_GEMM_MMA_FULL, abort_flag)) {
                        stop = true;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = ad0 + (uint64_t)(s * (p.a_bytes >> 4)), bd = bd0 + (uint64_t)(s * (p.b_bytes >> 4));
                    const uint32_t d = tmem + (uint32_t)(pi * kPartialCols);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (PAIR) tc_mma_pair_f8_if(d, ad + 2u * j, bd + 2u * j, idesc, j > 0 ? 1u : 0u, leader);
                        else tc_mma_f8_if(d, ad + 2u * j, bd + 2u * j, idesc, j > 0 ? 1u : 0u, leader);
                    }
                    if (PAIR) {
                        tc_commit_pair_if(&empty[s], 0x3, leader);
                        tc_commit_pair_if(&pfull[pi], 0x3, leader);
                    } else {
                        tc_commit_if(&empty[s], leader);
                        tc_commit_if(&pfull[pi], leader);
                    }
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                    if (++pi == NP) {
                        pi = 0;
                        pph ^= 1u;
                    }
                }
            }
            if (PAIR) tc_commit_pair_if(mma_done, 0x3, leader);
            else tc_commit_if(mma_done, leader);
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ drain
        if (CH == 4) setmaxnreg_inc<kB128DrainRegs>();
        const int q = warp & 3;                       // TMEM lane quadrant
        const int half = (warp - 4) >> 2;
        const int n_chunks = p.bn / 32;
        const int c0 = half == 0 ? 0 : (n_chunks + 1) / 2;                          // this warp's chunks
        const int nc = half == 0 ? (n_chunks + 1) / 2 : n_chunks - (n_chunks + 1) / 2;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(32 * c0);
        uint8_t *bufs = staging + (warp - 4) * 2 * kEpiChunkBytes;
        const uint32_t pempty0 = PAIR ? mapa_shared(smem_u32(&pempty[0]), 0) : 0u;
        const int last_sb = (p.N + 127) / 128 - 1;
        B128Tiles<GROUPED> tiles(p, lane);
        int pi = 0;
        uint32_t pph = 0, nstore = 0;
        bool stop = false;
        B128Tile t;
        for (int i = worker; !stop && tiles.at(i, t); i += workers) {
            const int m0q = t.row0 + (PAIR ? 128 * (int)rank : 0) + 32 * q;
            const int row_end = min(t.row_end, t.row0 + (1 << p.bm_shift));
            const bool any = m0q < row_end;           // warp-uniform
            const int row = m0q + lane;
            // the (at most two) 128-column scale blocks under this warp's columns
            const int nb0 = (t.n0 + 32 * c0) >> 7;
            const int split = (4 * (nb0 + 1)) - ((t.n0 >> 5) + c0);   // chunks in the first of them
            const float *sa = p.sa + row;
            const float *sb0 = p.sb + (int64_t)t.group * p.sb_step + (int64_t)min(nb0, last_sb) * p.num_kb;
            const float *sb1 = p.sb + (int64_t)t.group * p.sb_step + (int64_t)min(nb0 + 1, last_sb) * p.num_kb;
            const bool row_ok = row < row_end;
            uint64_t acc[CH * 16];
#pragma unroll
            for (int c = 0; c < CH * 16; ++c) acc[c] = 0u;
            // scales are fetched four blocks ahead of their use
            float f0[4], f1[4];
            auto fetch = [&](int kb, float &a, float &b) {
                a = b = 0.0f;
                if (row_ok && kb < p.num_kb) {
                    const float s = __ldg(sa + (int64_t)kb * p.sa_pitch);
                    a = s * __ldg(sb0 + kb);
                    b = s * __ldg(sb1 + kb);
                }
            };
#pragma unroll
            for (int j = 0; j < 4; ++j) fetch(j, f0[j], f1[j]);
            for (int kb0 = 0; kb0 < p.num_kb && !stop; kb0 += 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (kb0 + j < p.num_kb) {
                        if (!mbar_wait_bounded(&pfull[pi], pph, p.wait_limit_ns, SITE_GEMM_EPI_ACC, abort_flag)) {
                            stop = true;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t F0 = pk2(f0[j], f0[j]), F1 = pk2(f1[j], f1[j]);
                        const uint32_t t_p = t_lane + (uint32_t)(pi * kPartialCols);
                        auto release = [&] {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                if (PAIR) mbar_arrive_cluster(pempty0 + 8u * (uint32_t)pi);
                                else mbar_arrive(&pempty[pi]);
                            }
                        };
#pragma unroll
                        for (int h = 0; h < CH / 2; ++h) {
                            uint32_t r[2][32];
                            const bool on0 = any && 2 * h < nc, on1 = any && 2 * h + 1 < nc;   // warp-uniform
                            if (on0) tmem_ld32(t_p + 64 * h, r[0]);
                            if (on1) tmem_ld32(t_p + 64 * h + 32, r[1]);
                            if (on0) tmem_wait_ld();
                            if (h == CH / 2 - 1) release();
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                if (e == 0 ? on0 : on1) {
                                    const uint64_t F = 2 * h + e < split ? F0 : F1;
#pragma unroll
                                    for (int c = 0; c < 16; ++c)
                                        acc[32 * h + 16 * e + c] =
                                            fma2(pk2(__uint_as_float(r[e][2 * c]), __uint_as_float(r[e][2 * c + 1])), F,
                                                 acc[32 * h + 16 * e + c]);
                                }
                            }
                        }
                        if (++pi == NP) {
                            pi = 0;
                            pph ^= 1u;
                        }
                        fetch(kb0 + j + 4, f0[j], f1[j]);
                    }
                }
            }
            if (stop || !any) continue;
            // -------------------------------------------------------- epilogue
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                const int col = t.n0 + 32 * (c0 + ch);
                if (ch < nc && col < p.N) {
                    uint32_t packed[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float x0, x1;
                        upk2(acc[16 * ch + c], x0, x1);
                        if (p.epilogue == 1) gelu_erf2(x0, x1);
                        const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
                        packed[c] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    b128_store_chunk(p, &tmC, packed, m0q, row_end, col, lane, bufs, nstore);
                }
            }
        }
        if (lane == 0) bulk_wait_group_all();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        // every MMA (of the pair) has completed once mma_done has fired
        mbar_wait_bounded(mma_done, 0, p.wait_limit_ns, SITE_GEMM_TAIL, nullptr);
        if (PAIR) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
    griddep_launch_dependents();
    if (PAIR) cluster_sync();
}

}  // namespace mx
