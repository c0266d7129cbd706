// Linear layer of a few tokens on 4-bit weight codes with group scales, and its gated
// form (gate and up codes, the activation and the product): the decoding path.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gated_act.cuh"
#include "quest_internal.h"

namespace quest {

// y[0..n) = 0 (tc_host.cu).
cudaError_t launch_zero_fill(uint16_t* y, int32_t* acc, int64_t n, cudaStream_t stream);

namespace {

// ---------------------------------------------------------------------------
//   xt = H x / sqrt(had) per had-block (or x itself),  y[m][n] = sum_g Delta[n][g] sum_{k in g} v[n][k] xt[m][k]
// with v = q + 1/2 (midrise INT4) or the E2M1 value. At these token counts the layer is a read of the codes
// (K / 2 bytes a row and 4 bytes of scale per 128 columns), so every code byte is read once, 16 bytes a
// lane, straight into the fragment of an m16n8k16 MMA: 16 weight rows by 8 tokens, fp32 sums. (tcgen05 would
// need the decoded weights in shared memory and at least 64 rows of them; its rate is of no use here.)
//
// Columns may be permuted freely as long as both operands agree. Lane (g, t) of a warp reads the 32
// codes 32t .. 32t+31 of a 128-column group of rows g and g + 8: four words each, two MMAs per
// word. Midrise codes become fp16 with two logic operations a pair: nibble i and nibble i + 4
// of a word land in the mantissa of 16.0, giving 16 + (q + 8) = (q + 1/2) + 23.5, and 23.5 sum(xt) is
// taken off once per group (the offset is 3 times the largest value, which costs 2 of the sum's 24 bits).
// E2M1 codes become fp16 by the hardware conversion.
//
// xt is rounded to fp16 after scaling each token's group by a power of two that puts its largest value
// into [2^14, 2^15): 11 significant bits, half a unit 2^-12 of the value, 8 times below the
// rounding of the bf16 result, without overflow for any finite x.
//
// Work split: a cluster of CTAs cuts K, so that each CTA transforms and holds only its slice of x; inside
// a CTA the warps cut the rows and, where rows are few, K once more. Partial sums meet in shared
// memory and are added over the cluster in a fixed order.
constexpr int kLThreads = 256, kLWarps = 8;
constexpr int kGroup = 128;
constexpr int kMaxCluster = 8;

struct LowbitParams {
    const __nv_bfloat16* x;
    int64_t ld_x;
    const uint8_t* codes[2];
    const float* scales[2];
    __nv_bfloat16* y;
    int M, N, K, had;
    int groups;          // K / 128
    int scale_groups;    // scales per row: groups or 1
    int slice;           // groups per CTA of the cluster
    int wk;              // warps along K
    int tiles_per_warp;  // 16-row tiles
    float had_scale;     // 1 / sqrt(had)
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The four fp16 pairs of a word of eight codes.
template <bool FP4>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&p)[4]) {
    if constexpr (FP4) {
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
            : "r"(w));
    } else {
        // two's complement nibble to offset binary (flip its top bit, bit 9) under the exponent of 16.0
        constexpr uint32_t kMask = 0x03C003C0u, kFlip = 0x4C004C00u ^ 0x02000200u;
        p[0] = ((w << 6) & kMask) ^ kFlip;
        p[1] = ((w << 2) & kMask) ^ kFlip;
        p[2] = ((w >> 2) & kMask) ^ kFlip;
        p[3] = ((w >> 6) & kMask) ^ kFlip;
    }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// One 128-column group of one token, four columns a lane: butterflies of the blocks of
// `had` columns inside it (had <= 128; the stage across two groups is the caller's).
__device__ __forceinline__ void fwht_group(float (&v)[4], int had, int lane) {
    if (had >= 2) {
        const float a = v[0] + v[1], b = v[0] - v[1], c = v[2] + v[3], d = v[2] - v[3];
        v[0] = a + c; v[1] = b + d; v[2] = a - c; v[3] = b - d;   // had >= 16: both stages inside a lane
    }
#pragma unroll
    for (int h = 1; h < 32; h <<= 1) {
        if (4 * h < had) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float o = __shfl_xor_sync(0xFFFFFFFFu, v[j], h);
                v[j] = lane & h ? o - v[j] : v[j] + o;
            }
        }
    }
}

// Rounds one token's group to scaled fp16 and stores it as B fragments (16 bytes per (word of eight
// columns, lane t)), with the group's offset term and the scale's inverse.
template <bool FP4>
__device__ __forceinline__ void store_group(const float (&v)[4], int lane, uint8_t* frag, int tokens, int m, float2* meta) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const uint32_t e = max(top >> 23, 20u);   // (values below 2^-107 fade into zeros)
    const float mul = __uint_as_float((268u - e) << 23), inv = __uint_as_float((e - 14u) << 23);
    const uint32_t w0 = pack_f16(v[0] * mul, v[1] * mul), w1 = pack_f16(v[2] * mul, v[3] * mul);
    const int t = lane >> 3, w = (lane & 7) >> 1;
    uint8_t* at = frag + (w * tokens + m) * 64 + t * 16;
    float corr = 0.0f;
    if constexpr (FP4) {
        *reinterpret_cast<uint2*>(at + (lane & 1) * 8) = make_uint2(w0, w1);
    } else {
        // column order 0 4 1 5 2 6 3 7: the even lane holds columns 0-3, its neighbour 4-7
        const uint32_t o0 = __shfl_xor_sync(0xFFFFFFFFu, w0, 1), o1 = __shfl_xor_sync(0xFFFFFFFFu, w1, 1);
        if ((lane & 1) == 0)
            *reinterpret_cast<uint4*>(at) = make_uint4(__byte_perm(w0, o0, 0x5410), __byte_perm(w0, o0, 0x7632),
                                                       __byte_perm(w1, o1, 0x5410), __byte_perm(w1, o1, 0x7632));
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&w0));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&w1));
        corr = (f0.x + f0.y) + (f1.x + f1.y);
#pragma unroll
        for (int h = 16; h; h >>= 1) corr += __shfl_xor_sync(0xFFFFFFFFu, corr, h);
        corr *= 23.5f;
    }
    if (lane == 0) meta[m] = make_float2(corr, inv);
}

template <bool FP4, int NT, bool GATED, int ACT>
__global__ void __launch_bounds__(kLThreads, 2) lowbit_kernel(const LowbitParams p) {
    extern __shared__ __align__(16) uint8_t lsmem[];
    constexpr int MATS = GATED ? 2 : 1, TOK = 8 * NT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank, cs;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
    const int cluster = blockIdx.x / cs;
    const int m0 = blockIdx.y * TOK;
    const int tokens = min(TOK, p.M - m0);
    const int g0 = int(rank) * p.slice, g1 = min(g0 + p.slice, p.groups);
    const int wr = kLWarps / p.wk, wrow = warp / p.wk, wkk = warp % p.wk;
    const int row_tiles = wr * p.tiles_per_warp;   // per cluster
    // shared memory: B fragments [slice][4 words][tokens][64], meta [slice][TOK], partial sums
    // [wk][row_tiles][MATS][16][TOK]
    uint8_t* frags = lsmem;
    float2* meta = reinterpret_cast<float2*>(lsmem + size_t(p.slice) * tokens * 256);
    float* part = reinterpret_cast<float*>(meta + p.slice * TOK);

    pdl_wait();
    pdl_trigger();

    // ---- the CTA's slice of x
    if (p.had == 256) {
        const int pairs = (g1 - g0) / 2;
        for (int i = warp; i < pairs * tokens; i += kLWarps) {
            const int m = i / pairs, gp = 2 * (i % pairs);
            const __nv_bfloat16* src = p.x + (m0 + m) * p.ld_x + (g0 + gp) * kGroup + 4 * lane;
            const uint2 r0 = *reinterpret_cast<const uint2*>(src), r1 = *reinterpret_cast<const uint2*>(src + kGroup);
            float a[4] = {__uint_as_float(r0.x << 16), __uint_as_float(r0.x & 0xFFFF0000u),
                          __uint_as_float(r0.y << 16), __uint_as_float(r0.y & 0xFFFF0000u)};
            float b[4] = {__uint_as_float(r1.x << 16), __uint_as_float(r1.x & 0xFFFF0000u),
                          __uint_as_float(r1.y << 16), __uint_as_float(r1.y & 0xFFFF0000u)};
            fwht_group(a, 128, lane);
            fwht_group(b, 128, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float s = (a[j] + b[j]) * p.had_scale, d = (a[j] - b[j]) * p.had_scale;
                a[j] = s;
                b[j] = d;
            }
            store_group<FP4>(a, lane, frags + size_t(gp) * tokens * 256, tokens, m, meta + gp * TOK);
            store_group<FP4>(b, lane, frags + size_t(gp + 1) * tokens * 256, tokens, m, meta + (gp + 1) * TOK);
        }
    } else {
        const int ng = g1 - g0;
        for (int i = warp; i < ng * tokens; i += kLWarps) {
            const int m = i / ng, g = i % ng;
            const uint2 r = *reinterpret_cast<const uint2*>(p.x + (m0 + m) * p.ld_x + (g0 + g) * kGroup + 4 * lane);
            float v[4] = {__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u),
                          __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u)};
            if (p.had) {
                fwht_group(v, p.had, lane);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] *= p.had_scale;
            }
            store_group<FP4>(v, lane, frags + size_t(g) * tokens * 256, tokens, m, meta + g * TOK);
        }
    }
    __syncthreads();

    // ---- row tiles
    const int lg = lane >> 2, lt = lane & 3;
    int bm[NT];   // B column of the lane: a token that exists (what the others compute is dropped)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) bm[nt] = min(nt * 8 + lg, tokens - 1);
    for (int ti = 0; ti < p.tiles_per_warp; ++ti) {
        const int slot = ti * wr + wrow;
        const int64_t tile = int64_t(cluster) * row_tiles + slot;
        float total[MATS][NT][4] = {};
        if (tile * 16 < p.N) {
            const int64_t r0 = tile * 16 + lg, r1 = min(r0 + 8, int64_t(p.N) - 1);
            for (int g = g0 + wkk; g < g1; g += p.wk) {
                const uint8_t* fg = frags + size_t(g - g0) * tokens * 256 + lt * 16;
                const float2* mg = meta + (g - g0) * TOK;
                uint4 q0[MATS], q1[MATS];
                float s0[MATS], s1[MATS];
#pragma unroll
                for (int w = 0; w < MATS; ++w) {
                    const uint8_t* c = p.codes[w] + g * 64 + lt * 16;
                    q0[w] = __ldcs(reinterpret_cast<const uint4*>(c + r0 * (p.K / 2)));
                    q1[w] = __ldcs(reinterpret_cast<const uint4*>(c + r1 * (p.K / 2)));
                    const int sg = p.scale_groups == 1 ? 0 : g;
                    s0[w] = __ldg(p.scales[w] + r0 * p.scale_groups + sg);
                    s1[w] = __ldg(p.scales[w] + r1 * p.scale_groups + sg);
                }
                float acc[MATS][NT][4] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 b[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        b[nt] = *reinterpret_cast<const uint4*>(fg + (j * tokens + bm[nt]) * 64);
#pragma unroll
                    for (int w = 0; w < MATS; ++w) {
                        uint32_t pa[4], pb[4];
                        decode8<FP4>(j == 0 ? q0[w].x : j == 1 ? q0[w].y : j == 2 ? q0[w].z : q0[w].w, pa);
                        decode8<FP4>(j == 0 ? q1[w].x : j == 1 ? q1[w].y : j == 2 ? q1[w].z : q1[w].w, pb);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_16816(acc[w][nt], pa[0], pb[0], pa[1], pb[1], b[nt].x, b[nt].y);
                            mma_16816(acc[w][nt], pa[2], pb[2], pa[3], pb[3], b[nt].z, b[nt].w);
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 ma = mg[nt * 8 + 2 * lt], mb = mg[nt * 8 + 2 * lt + 1];
#pragma unroll
                    for (int w = 0; w < MATS; ++w) {
                        total[w][nt][0] = fmaf(s0[w] * ma.y, acc[w][nt][0] - ma.x, total[w][nt][0]);
                        total[w][nt][1] = fmaf(s0[w] * mb.y, acc[w][nt][1] - mb.x, total[w][nt][1]);
                        total[w][nt][2] = fmaf(s1[w] * ma.y, acc[w][nt][2] - ma.x, total[w][nt][2]);
                        total[w][nt][3] = fmaf(s1[w] * mb.y, acc[w][nt][3] - mb.x, total[w][nt][3]);
                    }
                }
            }
        }
        float* dst = part + (size_t(wkk) * row_tiles + slot) * (MATS * 16 * TOK);
#pragma unroll
        for (int w = 0; w < MATS; ++w)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                *reinterpret_cast<float2*>(dst + (w * 16 + lg) * TOK + nt * 8 + 2 * lt) =
                    make_float2(total[w][nt][0], total[w][nt][1]);
                *reinterpret_cast<float2*>(dst + (w * 16 + lg + 8) * TOK + nt * 8 + 2 * lt) =
                    make_float2(total[w][nt][2], total[w][nt][3]);
            }
    }

    // ---- sum over the cluster and the K warps, in rank and warp order
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    const uint32_t part_addr = static_cast<uint32_t>(__cvta_generic_to_shared(part));
    const int outs = row_tiles * 16 * tokens;
    for (int i = int(rank) * kLThreads + threadIdx.x; i < outs; i += int(cs) * kLThreads) {
        const int r = i % (row_tiles * 16), m = i / (row_tiles * 16);
        const int64_t n = int64_t(cluster) * row_tiles * 16 + r;
        if (n >= p.N) continue;
        float v[MATS] = {};
        for (uint32_t c = 0; c < cs; ++c) {
            uint32_t base;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base) : "r"(part_addr), "r"(c));
            for (int k = 0; k < p.wk; ++k)
#pragma unroll
                for (int w = 0; w < MATS; ++w) {
                    float f;
                    const uint32_t off = uint32_t((((k * row_tiles + r / 16) * MATS + w) * 16 + r % 16) * TOK + m) * 4;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(base + off) : "memory");
                    v[w] += f;
                }
        }
        float out = v[0];
        if constexpr (GATED) out = v[0] * gate_sigmoid<ACT>(v[0]) * v[1];
        p.y[int64_t(m0 + m) * p.N + n] = __float2bfloat16_rn(out);
    }
    // no CTA leaves while another may still read its partial sums
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <bool FP4, int NT, bool GATED, int ACT>
cudaError_t launch_one(const LowbitArgs& a, cudaStream_t stream) {
    constexpr int MATS = GATED ? 2 : 1, TOK = 8 * NT;
    LowbitParams p;
    p.x = reinterpret_cast<const __nv_bfloat16*>(a.x);
    p.ld_x = a.ld_x;
    for (int w = 0; w < 2; ++w) {
        p.codes[w] = a.codes[w];
        p.scales[w] = a.scales[w];
    }
    p.y = reinterpret_cast<__nv_bfloat16*>(a.y);
    p.M = (int)a.M; p.N = (int)a.N; p.K = (int)a.K; p.had = a.had;
    p.groups = (int)(a.K / kGroup);
    p.scale_groups = a.scale_groups;
    p.had_scale = a.had ? (float)(1.0 / sqrt((double)a.had)) : 1.0f;
    const int tokens = p.M < TOK ? p.M : TOK, token_tiles = (p.M + TOK - 1) / TOK;
    const int sms = sm_count();
    const int unit = a.had == 256 ? 2 : 1;   // groups that stay together
    // cluster: the fewest CTAs along K whose slice of x stays within 48 KB of shared memory
    int cs = 1;
    auto slice_of = [&](int c) { return ((p.groups + c - 1) / c + unit - 1) / unit * unit; };
    while (cs < kMaxCluster && slice_of(cs) * tokens * 256 > 48 * 1024) cs *= 2;
    p.slice = slice_of(cs);
    // warps along K until every SM has 16 warps' worth of tiles
    const int64_t tiles = (p.N + 15) / 16;
    p.wk = 1;
    while (p.wk < kLWarps && p.wk < p.slice && tiles * cs * p.wk < int64_t(sms) * 16) p.wk *= 2;
    const size_t xbytes = size_t(p.slice) * tokens * 256 + size_t(p.slice) * TOK * 8;
    const size_t tile_bytes = size_t(kLWarps) * MATS * 16 * TOK * 4;   // partial sums of one tile per warp
    // tiles per warp: about two CTAs an SM in one wave, within the shared memory
    const int wr = kLWarps / p.wk;
    int64_t tpw = (tiles * cs * token_tiles + int64_t(wr) * sms * 2 - 1) / (int64_t(wr) * sms * 2);
    const size_t room = (xbytes > 100 * 1024 ? 220 * 1024 : 110 * 1024) - xbytes;
    if (tpw > int64_t(room / tile_bytes)) tpw = int64_t(room / tile_bytes);
    if (tpw < 1) tpw = 1;
    p.tiles_per_warp = (int)tpw;
    const size_t smem = xbytes + tile_bytes * tpw;
    const int64_t clusters = (tiles + wr * tpw - 1) / (wr * tpw);

    auto kernel = lowbit_kernel<FP4, NT, GATED, ACT>;
    static thread_local int attr_dev = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (attr_dev != dev) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        attr_dev = dev;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * cs), (unsigned)token_tiles);
    cfg.blockDim = dim3(kLThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool FP4, bool GATED, int ACT>
cudaError_t launch_tokens(const LowbitArgs& a, cudaStream_t stream) {
    return a.M <= 8 ? launch_one<FP4, 1, GATED, ACT>(a, stream) : launch_one<FP4, 2, GATED, ACT>(a, stream);
}

template <bool FP4>
cudaError_t launch_grid(const LowbitArgs& a, cudaStream_t stream) {
    if (!a.codes[1]) return launch_tokens<FP4, false, QUEST_ACT_SILU>(a, stream);
    return a.act == QUEST_ACT_SILU ? launch_tokens<FP4, true, QUEST_ACT_SILU>(a, stream)
                                   : launch_tokens<FP4, true, QUEST_ACT_GELU_TANH>(a, stream);
}

}  // namespace

cudaError_t launch_lowbit(const LowbitArgs& a, cudaStream_t stream) {
    if (a.M == 0 || a.N == 0) return cudaSuccess;
    if (a.K == 0) return launch_zero_fill(a.y, nullptr, a.M * a.N, stream);
    return a.fp4 ? launch_grid<true>(a, stream) : launch_grid<false>(a, stream);
}

}  // namespace quest
