// Gated feed-forward block, forward: both projections, the activation, the product
// and the 8-bit checkpoint of the projections in one CTA-pair tcgen05 kernel.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace quest {
namespace {
// Device-side status word of this file's kernels (0 = fine). Written only when a
// bounded wait gives up; read and cleared by quest_device_status().
__device__ int g_tc_status = 0;
}  // namespace
}  // namespace quest

#include "gated_act.cuh"
#include "tc_common.cuh"

namespace quest {
namespace {

// ---------------------------------------------------------------------------
//   a[m][f] = sum_k x[m][k] wg[f][k],  b[m][f] = sum_k x[m][k] wu[f][k]    (bf16, fp32 sums)
//   h[m][f] = act(a) b                                                     (bf16)
// and, for training, the checkpoint of a and b: int8 codes and a step per 128 columns.
//
// One MMA of the pair is M = 256, N = 256, K = 16; its B operand is the even CTA's 128 rows
// followed by the odd CTA's. The even CTA loads 128 rows of wg and the odd CTA the same 128
// rows of wu, so the accumulator holds a in columns 0-127 and b in columns 128-255 of the same 128
// outputs: the thread that owns an accumulator row has both in reach, and a and b never go
// to HBM unless as 8-bit codes. A checkpoint group is exactly the tile's 128 columns, so its
// maximum is a loop over registers with no exchange between threads.
constexpr uint32_t kIdescBf16Pair = (1u << 4)     // D: fp32
                                  | (1u << 7)     // A: bf16
                                  | (1u << 10)    // B: bf16
                                  | (uint32_t(BN >> 3) << 17) | (uint32_t(256 >> 4) << 24);

__device__ __forceinline__ void tc_mma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(kIdescBf16Pair), "r"(accumulate)
        : "memory");
}

// Shared memory per CTA: the operand ring of the pair kernels, then two staging sets of
// 32 columns: h (64-byte rows), codes of a and of b (32-byte rows), then the barriers.
constexpr uint32_t kGSetBytes = kCBytes + 2 * BM * kChunkCols;
constexpr uint32_t kGSmemC = kPSmemB + kPStages * kPStageB;
constexpr uint32_t kGSmemBar = kGSmemC + 2 * kGSetBytes;
constexpr uint32_t kGSmemTmemSlot = kGSmemBar + kPNumBars * 8;
constexpr uint32_t kGSmemAbort = kGSmemTmemSlot + 4;
constexpr uint32_t kGSmemTotal = kGSmemAbort + 4 + 1024;
static_assert(kGSmemTotal <= 227 * 1024, "gated kernel shared memory");

constexpr int kCols = 128;   // outputs per tile: half the accumulator's columns

struct GatedParams {
    float* scales;              // [M, 2 groups] checkpoint steps
    int M, F, groups;           // groups = ceil(F / 128)
    int num_m2, num_f, num_k;   // 256-row tiles, 128-output tiles, 64-element steps of K
};

template <int ACT, bool CKPT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gated_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_wg,
                  const __grid_constant__ CUtensorMap map_wu, const __grid_constant__ CUtensorMap map_h,
                  const __grid_constant__ CUtensorMap map_ca, const __grid_constant__ CUtensorMap map_cb,
                  const GatedParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = sbase + kGSmemBar;                 // [kPStages], used in the even CTA
    const uint32_t bar_empty = bar_full + 8 * kPStages;          // [kPStages]
    const uint32_t bar_tfull = bar_empty + 8 * kPStages;         // [2]
    const uint32_t bar_tempty = bar_tfull + 16;                  // [2], used in the even CTA
    const uint32_t bar_drain = bar_tempty + 16;                  // [1]
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kGSmemAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kGSmemTmemSlot);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool even = rank == 0;
    const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
    const int num_tiles = p.num_m2 * p.num_f;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPStages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, 2);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            const uint32_t full_even = map_to_rank(bar_full, 0);
            const CUtensorMap* map_w = even ? &map_wg : &map_wu;
            uint32_t stage = 0, phase = 0;
            uint64_t issued = 0;
            bool ok = true;
            for (int tile = pair; tile < num_tiles && ok; tile += num_pairs) {
                const int m0 = (tile / p.num_f) * 256 + 128 * int(rank);
                const int f0 = (tile % p.num_f) * kCols;
                for (int kb = 0; kb < p.num_k; ++kb) {
                    if (!mbar_wait(bar_empty + 8 * stage, phase ^ 1, abort_flag, kWaitLimitNs, kSuspendProducerNs)) {
                        ok = false;
                        break;
                    }
                    if (even) mbar_arrive_expect_tx(bar_full + 8 * stage, kPTxBytes);
                    const uint32_t fb = full_even + 8 * stage;
                    tma_load_2d_pair(sbase + kPSmemA + stage * kPStageA, &map_x, kb * 64, m0, fb);
                    tma_load_2d_pair(sbase + kPSmemB + stage * kPStageB, map_w, kb * 64, f0, fb);
                    ++issued;
                    if (++stage == kPStages) { stage = 0; phase ^= 1; }
                }
            }
            // giving up: no CTA may leave while a copy into its shared memory is in flight
            if (!ok && even) {
                const uint64_t n = issued < kPStages ? issued : kPStages;
                for (uint64_t i = issued - n; i < issued; ++i) {
                    const uint32_t st = uint32_t(i % kPStages), ph = uint32_t((i / kPStages) & 1);
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(bar_full + 8 * st, ph) && global_timer_ns() - t0 < kWaitLimitNs) {
                    }
                }
            } else if (!ok) {
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 10000000ull) {
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (even CTA)
        if (even && lane == 0) {
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            int local = 0;
            for (int tile = pair; tile < num_tiles && ok; tile += num_pairs, ++local) {
                const uint32_t buf = local & 1, bphase = (local >> 1) & 1;
                if (!mbar_wait(bar_tempty + 8 * buf, bphase ^ 1, abort_flag, kWaitLimitNs, kSuspendMmaNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + buf * BN;
                for (int kb = 0; kb < p.num_k; ++kb) {
                    if (!mbar_wait(bar_full + 8 * stage, phase, abort_flag, kWaitLimitNs, kSuspendMmaNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = sbase + kPSmemA + stage * kPStageA;
                    const uint32_t b_addr = sbase + kPSmemB + stage * kPStageB;
#pragma unroll
                    for (int kk = 0; kk < BK / kUmmaK; ++kk) {
                        tc_mma_bf16_pair(d_tmem, smem_desc_k128(a_addr + kk * kUmmaK),
                                         smem_desc_k128(b_addr + kk * kUmmaK), (kb | kk) != 0);
                    }
                    tc_commit_pair_mc(bar_empty + 8 * stage);
                    if (++stage == kPStages) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                tc_commit_pair_mc(bar_tfull + 8 * buf);
            }
            tc_commit_pair(bar_drain);
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(bar_drain, 0) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue (warps 2..5, both CTAs)
        const int et = threadIdx.x - 64;
        const int quarter = warp & 3;
        const int row_in_tile = quarter * 32 + lane;
        const uint32_t lane_addr = uint32_t(quarter * 32) << 16;
        const uint32_t tempty_even = map_to_rank(bar_tempty, 0);
        int local = 0;
        int cbuf = 0;
        for (int tile = pair; tile < num_tiles; tile += num_pairs, ++local) {
            const int m0 = (tile / p.num_f) * 256 + 128 * int(rank);
            const int ft = tile % p.num_f, f0 = ft * kCols;
            const uint32_t buf = local & 1, bphase = (local >> 1) & 1;
            const int m = m0 + row_in_tile;
            const bool got = mbar_wait(bar_tfull + 8 * buf, bphase, abort_flag, kWaitLimitNs, kSuspendEpilogueNs);
            if (epi_any(!got)) break;
            tc_fence_after();
            const uint32_t t_a = tmem_base + lane_addr + buf * BN, t_b = t_a + kCols;
            CkptScale sa = {0.0f, 0.0f}, sb = {0.0f, 0.0f};
            if constexpr (CKPT) {
                // the group's maxima: columns past F are zero (their weight rows read as zero)
                uint32_t ma = 0, mb = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t ra[32], rb[32];
                    QUEST_TMEM_LD32(t_a + 32 * c, ra);
                    QUEST_TMEM_LD32(t_b + 32 * c, rb);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        ma = max(ma, ra[i] & 0x7FFFFFFFu);
                        mb = max(mb, rb[i] & 0x7FFFFFFFu);
                    }
                }
                sa = ckpt_scale(ma);
                sb = ckpt_scale(mb);
                if (m < p.M) {
                    float* row = p.scales + int64_t(m) * (2 * p.groups) + ft;
                    row[0] = sa.delta;
                    row[p.groups] = sb.delta;
                }
            }
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                if (m0 >= p.M || f0 + c * kChunkCols >= p.F) break;   // nothing of this chunk is stored (uniform)
                uint32_t ra[32], rb[32];
                QUEST_TMEM_LD32(t_a + 32 * c, ra);
                QUEST_TMEM_LD32(t_b + 32 * c, rb);
                tmem_wait_ld();
                const uint32_t set = sbase + kGSmemC + cbuf * kGSetBytes;
                const uint32_t stg = set + row_in_tile * (kChunkCols * 2);
                const uint32_t swz = (row_in_tile >> 1) & 3;
#pragma unroll
                for (int q16 = 0; q16 < 4; ++q16) {
                    uint32_t o[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int i = 8 * q16 + 2 * w;
                        const float a0 = __uint_as_float(ra[i]), a1 = __uint_as_float(ra[i + 1]);
                        const float b0 = __uint_as_float(rb[i]), b1 = __uint_as_float(rb[i + 1]);
                        o[w] = pack_bf16(a0 * gate_sigmoid<ACT>(a0) * b0, a1 * gate_sigmoid<ACT>(a1) * b1);
                    }
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stg + ((q16 ^ swz) << 4)), "r"(o[0]),
                                 "r"(o[1]), "r"(o[2]), "r"(o[3])
                                 : "memory");
                }
                if constexpr (CKPT) {
                    const uint32_t ca = set + kCBytes + row_in_tile * kChunkCols, cb = ca + BM * kChunkCols;
                    const uint32_t swz32 = (row_in_tile >> 2) & 1;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        uint32_t qa[4], qb[4];
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const int i = 16 * hf + 4 * w;
                            qa[w] = ckpt_pack4(__uint_as_float(ra[i]), __uint_as_float(ra[i + 1]),
                                               __uint_as_float(ra[i + 2]), __uint_as_float(ra[i + 3]), sa.inv);
                            qb[w] = ckpt_pack4(__uint_as_float(rb[i]), __uint_as_float(rb[i + 1]),
                                               __uint_as_float(rb[i + 2]), __uint_as_float(rb[i + 3]), sb.inv);
                        }
                        const uint32_t off = (hf ^ swz32) << 4;
                        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(ca + off), "r"(qa[0]), "r"(qa[1]),
                                     "r"(qa[2]), "r"(qa[3])
                                     : "memory");
                        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(cb + off), "r"(qb[0]), "r"(qb[1]),
                                     "r"(qb[2]), "r"(qb[3])
                                     : "memory");
                    }
                }
                fence_proxy_async_smem();
                epi_bar();
                if (et == 0) {
                    const int col = f0 + c * kChunkCols;
                    tma_store_2d(&map_h, set, col, m0);
                    if constexpr (CKPT) {
                        tma_store_2d(&map_ca, set + kCBytes, col, m0);
                        tma_store_2d(&map_cb, set + kCBytes + BM * kChunkCols, col, m0);
                    }
                    bulk_commit();
                    bulk_wait_read_le1();
                }
                epi_bar();
                cbuf ^= 1;
            }
            tc_fence_before();
            epi_bar();
            if (et == 0) mbar_arrive_remote(tempty_even + 8 * buf);
        }
        if (et == 0) bulk_wait_all();
    }

    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols)
                     : "memory");
    }
}

template <int ACT, bool CKPT>
cudaError_t launch_pair(const GatedArgs& g, cudaStream_t stream) {
    CUtensorMap mx, mg, mu, mh, ma, mb;
    if (!make_map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.x, g.K, g.M, g.K * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_2d(&mg, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.wg, g.K, g.F, g.K * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_2d(&mu, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.wu, g.K, g.F, g.K * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_2d(&mh, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.h, g.F, g.M, g.F * 2, kChunkCols, 128,
                     CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    ma = mb = mh;   // never used without a checkpoint
    if (CKPT && (!make_map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.codes, g.F, g.M, 2 * g.F, kChunkCols, 128,
                              CU_TENSOR_MAP_SWIZZLE_32B) ||
                 !make_map_2d(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.codes + g.F, g.F, g.M, 2 * g.F, kChunkCols, 128,
                              CU_TENSOR_MAP_SWIZZLE_32B)))
        return cudaErrorInvalidValue;
    GatedParams p;
    p.scales = g.scales;
    p.M = (int)g.M; p.F = (int)g.F;
    p.groups = (int)((g.F + 127) / 128);
    p.num_m2 = (int)((g.M + 255) / 256);
    p.num_f = p.groups;
    p.num_k = (int)((g.K + 63) / 64);
    static thread_local int attr_dev = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (attr_dev != dev) {
        cudaError_t e = cudaFuncSetAttribute(gated_pair_kernel<ACT, CKPT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmemTotal);
        if (e != cudaSuccess) return e;
        attr_dev = dev;
    }
    const int64_t tiles = int64_t(p.num_m2) * p.num_f;
    const int pairs = pair_clusters(dev, (const void*)gated_pair_kernel<ACT, CKPT>, kThreads, kGSmemTotal);
    const int grid_pairs = tiles < pairs ? (int)tiles : pairs;
    return launch_pdl(gated_pair_kernel<ACT, CKPT>, dim3(2 * grid_pairs), dim3(kThreads), kGSmemTotal, stream, mx, mg,
                      mu, mh, ma, mb, p);
}

// K == 0: both projections are empty sums, so h, the codes and the steps are all zero.
__global__ void gated_zero_kernel(uint16_t* h, int8_t* codes, float* scales, int64_t n, int64_t n_scales) {
    pdl_wait();
    pdl_trigger();
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        h[i] = 0;
        if (codes) codes[2 * i] = codes[2 * i + 1] = 0;
        if (codes && i < n_scales) scales[i] = 0.0f;
    }
}

}  // namespace

cudaError_t launch_gated_linear(const GatedArgs& g, cudaStream_t stream) {
    if (g.M == 0 || g.F == 0) return cudaSuccess;
    if (g.K == 0) {
        const int64_t n = g.M * g.F, blocks = (n + 255) / 256;   // n >= the number of steps: F >= 16, two per 128 columns
        return launch_pdl(gated_zero_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, g.h,
                          g.codes, g.scales, n, g.M * 2 * ((g.F + 127) / 128));
    }
    if (g.act == QUEST_ACT_SILU)
        return g.codes ? launch_pair<QUEST_ACT_SILU, true>(g, stream) : launch_pair<QUEST_ACT_SILU, false>(g, stream);
    return g.codes ? launch_pair<QUEST_ACT_GELU_TANH, true>(g, stream)
                   : launch_pair<QUEST_ACT_GELU_TANH, false>(g, stream);
}

int read_and_clear_gated_status(cudaStream_t stream, cudaError_t* err) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_tc_status, sizeof(int), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && v != 0)
        e = cudaMemcpyToSymbolAsync(g_tc_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    *err = e;
    return v;
}

}  // namespace quest
