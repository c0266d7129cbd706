// Linear layer of a few tokens on 4-bit weight codes with group scales, and its gated
// form (gate and up codes, the activation and the product): the decoding path.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

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
// lane, straight into MMA fragments: 16 weight rows by 8 tokens. (tcgen05 would need the decoded weights
// in shared memory and at least 64 rows of them; its rate is of no use here.) At HBM's rate an SM has 38 cycles
// per KB of codes, 76 instructions of the integer pipe and 18 MMAs, so the decoding decides the form:
//
// Midrise codes stay integers. Flipping a nibble's top bit gives u = q + 8 in 0..15; a word of eight codes
// becomes two fragment words of bytes with three instructions (as fp16 pairs it took eight). x is rounded to
// 16-bit fixed point under a scale per token and group, x = 256 hi + lo, and two m16n8k32 integer MMAs give
// sum(u hi) and sum(u lo) exactly; sum((q + 1/2) x) = sum(u x) - 7.5 sum(x) is exact too. The rounding of x is
// the only one before the scales: 2^-16 of the group's largest value.
//
// E2M1 codes become fp16 pairs by the hardware conversion (as fast as a logic instruction, two codes each)
// and take m16n8k16 with fp32 sums; x is rounded to fp16 under a power of two per token and group
// that puts its largest value into [2^14, 2^15): off by half a step, 2^-11 of each value, or where fp16 is
// subnormal 2^-25, which is 2^-39 of the largest.
//
// Columns may be permuted freely as long as both operands agree: lane (g, t) of a warp takes the 32
// codes 32t .. 32t+31 of a 128-column group of rows g and g + 8, and x's fragments are laid out to match.
// A group of a row is 64 bytes, half a line, and a load instruction whose lanes touch half lines of eight rows
// leaves the SM waiting on its requests (the loads alone, with scales: 54 us at 22016 x 8192 twice, 45 with whole
// lines, 35 once the scales went through shared memory; all of it 90 us and 54). So groups
// are loaded in pairs: an instruction takes the whole line of four rows, even lanes' rows the first
// group and odd lanes' rows the second, another instruction the neighbouring rows the other way round, and a
// select by the lane's parity sorts them. The second group's rows come out pairwise swapped; its sums
// are kept apart and swapped back once per tile.
//
// Work split. A cluster of `cs` CTAs cuts K, so that each CTA transforms and holds only its slice of
// x; clusters walk over the 16-row tiles. Inside a CTA, wk warps cut the slice and the
// remaining factor takes further row tiles. Every warp keeps its next kPairs pairs of groups in
// registers, loaded across tile boundaries and before x is transformed, so that memory never
// waits for a tile's end. Partial sums meet in shared memory and are added in warp and rank order.
constexpr int kGroup = 128;
constexpr int kMaxCluster = 8;
constexpr int kLowbitMaxK = 32768;   // as the callers check
constexpr int kChunk = 8;    // groups whose scales are fetched together
constexpr int kWarps = 16;   // one CTA an SM: x's slice is held once
static_assert((kWarps & (kWarps - 1)) == 0, "the warps along K must divide a CTA's warps: a row group's barrier counts them");

struct LowbitParams {
    const __nv_bfloat16* x;
    int64_t ld_x;
    uint8_t* staged;     // B fragments and their meta of all tokens, written by stage_kernel; null: each CTA's own work
    const uint8_t* codes[2];
    const float* scales[2];
    __nv_bfloat16* y;
    int M, N, K, had;
    int groups;          // K / 128
    int scale_groups;    // scales per row: groups or 1
    int slice;           // groups per CTA of the cluster (even, but for a single CTA's last)
    int wk;              // warps along K
    int iters;           // row tiles per warp
    int batch;           // of them, those whose sums a cluster collects at a time
    int clusters;
    float had_scale;     // 1 / sqrt(had)
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The four fp16 pairs of a word of eight E2M1 codes.
__device__ __forceinline__ void decode_e2m1(uint32_t w, uint32_t (&p)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(w));
}

// d += u s (bytes, unsigned times signed) and the unsigned form.
__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_u8u8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Butterflies over the 16 values of a lane (the low four bits of the column).
__device__ __forceinline__ void fwht16(float2 (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = make_float2(v[j].x + v[j].y, v[j].x - v[j].y);
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if ((j & h) == 0) {
                const float2 a = v[j], b = v[j + h];
                v[j] = __fadd2_rn(a, b);
                v[j + h] = __ffma2_rn(b, make_float2(-1.0f, -1.0f), a);
            }
        }
    }
}

// The 16 columns of x that this lane transforms in the step that begins with item `base` (see stage_x).
__device__ __forceinline__ void fetch_x(const LowbitParams& p, int m0, int items, int g0, int ng, int base,
                                        uint4 (&raw)[2]) {
    if (base >= items) return;
    const int lane = threadIdx.x & 31, item = min(base + (lane >> 3), items - 1);
    const int m = item / ng, g = item - m * ng;
    const uint4* src =
        reinterpret_cast<const uint4*>(p.x + (m0 + m) * p.ld_x + int64_t(g0 + g) * kGroup + 16 * (lane & 7));
    raw[0] = __ldg(src);
    raw[1] = __ldg(src + 1);
}

// A slice of x, transformed, as B fragments, by `warps` warps. Four (token, group) items a warp step, groups fastest,
// eight lanes an item, 16 columns a lane: two of the eight-column words that lane t = column / 32 of the MMA needs.
template <bool FP4, int TOK>
__device__ __forceinline__ void stage_x(const LowbitParams& p, int m0, int tokens, int g0, int ng, int warp, int warps,
                                        uint4 (&raw)[2], uint8_t* frags, float2* meta) {
    const int lane = threadIdx.x & 31, u = lane & 7;
    const int items = ng * tokens;
    // each step's x is read one step ahead, the first by the caller
    for (int base = warp * 4; base < items; base += warps * 4) {
        const bool live = base + (lane >> 3) < items;
        const int item = live ? base + (lane >> 3) : items - 1;   // (spare lanes only keep the shuffles whole)
        const int m = item / ng, g = item - m * ng;
        float2 v[8];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                // (taken down by 2^8, exactly, so that no sum of 256 finite values overflows; the group's scale makes it up)
                v[4 * c + j] = __fmul2_rn(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)),
                                          make_float2(0.00390625f, 0.00390625f));
        }
        fetch_x(p, m0, items, g0, ng, base + warps * 4, raw);
        if (p.had) {
            fwht16(v);
            // the stages between lanes: the lower lane keeps the sum, the upper one the difference (slices are
            // whole pairs of groups, so blocks of 256 lie in neighbouring items)
#pragma unroll 1
            for (int h = 1; 16 * h < p.had; h <<= 1) {
                const float sign = lane & h ? -1.0f : 1.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 o = make_float2(__shfl_xor_sync(0xFFFFFFFFu, v[j].x, h),
                                                 __shfl_xor_sync(0xFFFFFFFFu, v[j].y, h));
                    v[j] = __ffma2_rn(v[j], make_float2(sign, sign), o);
                }
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, max(__float_as_uint(v[j].x) & 0x7FFFFFFFu, __float_as_uint(v[j].y) & 0x7FFFFFFFu));
#pragma unroll
        for (int h = 1; h < 8; h <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, h));
        // word w of token m lies ((4 g + w) tokens + m) 64 bytes in: a fragment read is one run of bytes
        uint8_t* at = frags + (size_t(g) * 4 * tokens + m) * 64 + (u >> 1) * 16;
        const int w0 = 2 * (u & 1);
        float2 entry;
        uint4 out[2];
        if constexpr (FP4) {
            const uint32_t e = max(top >> 23, 20u);   // (groups below 2^-99 fade into zeros)
            const float mul = __uint_as_float((268u - e) << 23);
            entry = make_float2(0.0f, __uint_as_float((e - 14u) << 23) * (256.0f * p.had_scale));
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __half2 hv = __floats2half2_rn(v[4 * w + j].x * mul, v[4 * w + j].y * mul);
                    h[j] = *reinterpret_cast<const uint32_t*>(&hv);
                }
                out[w] = make_uint4(h[0], h[1], h[2], h[3]);
            }
        } else {
            // the group's largest value becomes 32767; a group below 2^-100 counts as zero
            const float amax = __uint_as_float(top);
            const bool zero = amax < 3.0814879110195774e-33f;   // (2^-108, after the 2^-8)
            const float mul = zero ? 0.0f : 32767.0f / amax;
            uint32_t sum = 0;   // (two's complement; a non-finite group's wraps)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                uint32_t b[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // 1.5 * 2^23 + x holds x, rounded to nearest, in its low 16 bits
                    const float2 f = __ffma2_rn(v[4 * w + j], make_float2(mul, mul), make_float2(12582912.0f, 12582912.0f));
                    b[2 * j] = __float_as_uint(f.x);
                    b[2 * j + 1] = __float_as_uint(f.y);
                    sum += b[2 * j] + b[2 * j + 1] - 2 * 0x4B400000u;
                }
                // columns 0 2 4 6 and 1 3 5 7: high bytes, then low bytes
                out[w] = make_uint4(__byte_perm(__byte_perm(b[0], b[2], 0x0051), __byte_perm(b[4], b[6], 0x0051), 0x5410),
                                    __byte_perm(__byte_perm(b[1], b[3], 0x0051), __byte_perm(b[5], b[7], 0x0051), 0x5410),
                                    __byte_perm(__byte_perm(b[0], b[2], 0x0040), __byte_perm(b[4], b[6], 0x0040), 0x5410),
                                    __byte_perm(__byte_perm(b[1], b[3], 0x0040), __byte_perm(b[5], b[7], 0x0040), 0x5410));
            }
#pragma unroll
            for (int h = 1; h < 8; h <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, h);
            // 15 sum(x), and half the step of x (a non-finite largest value makes it non-finite)
            entry = make_float2(__uint_as_float(15u * sum), zero ? 0.0f : amax * (p.had_scale * (128.0f / 32767.0f)));
        }
        if (!live) continue;
#pragma unroll
        for (int w = 0; w < 2; ++w) *reinterpret_cast<uint4*>(at + (w0 + w) * tokens * 64) = out[w];
        if (u == 0) meta[g * TOK + m] = entry;
    }
}

// The staged copy of x for token tile `tile`: fragments [groups][4 words][tokens][64], and meta [groups][TOK] behind all of them.
template <int TOK>
__device__ __forceinline__ uint8_t* staged_frags(const LowbitParams& p, int tile) {
    return p.staged + size_t(tile) * TOK * p.groups * 256;
}
template <int TOK>
__device__ __forceinline__ float2* staged_meta(const LowbitParams& p, int tile) {
    return reinterpret_cast<float2*>(p.staged + size_t(p.M) * p.groups * 256) + size_t(tile) * p.groups * TOK;
}

template <bool FP4, int TOK>
__global__ void __launch_bounds__(128) stage_kernel(const LowbitParams p) {
    pdl_wait();
    pdl_trigger();
    const int tile = blockIdx.y, m0 = tile * TOK, tokens = min(TOK, p.M - m0);
    const int warp = blockIdx.x * 4 + (threadIdx.x >> 5), warps = gridDim.x * 4;
    uint4 raw[2];
    fetch_x(p, m0, p.groups * tokens, 0, p.groups, warp * 4, raw);
    stage_x<FP4, TOK>(p, m0, tokens, 0, p.groups, warp, warps, raw, staged_frags<TOK>(p, tile), staged_meta<TOK>(p, tile));
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void* smem_dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(smem_dst))),
                 "l"(src), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copy16_async(void* smem_dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(smem_dst))),
                 "l"(src)
                 : "memory");
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// NT: tokens / 8.
template <bool FP4, int NT, bool GATED, int ACT>
__global__ void __launch_bounds__(kWarps * 32, 1) lowbit_kernel(const LowbitParams p) {
    extern __shared__ __align__(256) uint8_t lsmem[];
    constexpr int MATS = GATED ? 2 : 1, TOK = 8 * NT;
    // Pairs of groups in registers (of each matrix), and per turn of the loop, as registers allow. One matrix, up to 8
    // tokens: 44032 x 8192 took 61, 55 and 52 us with 1, 2 and 4; 16 tokens x 8192 x 22016: 45.6, 45.5 and 62. Two matrices:
    // 5 x 22016 x 8192 took 53 us with one of each, 60 with two.
    constexpr int kPairs = GATED ? 1 : NT == 1 ? 4 : 2;
    static_assert(kChunk % (2 * kPairs) == 0, "a turn lies in one chunk of scales");
    constexpr int kTile = MATS * TOK * 16;   // one tile's sums, [matrix][token][row]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank, cs;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
    const int cluster = blockIdx.x / cs;
    const int m0 = blockIdx.y * TOK;
    const int tokens = min(TOK, p.M - m0);
    const int g0 = int(rank) * p.slice, ng = max(min(p.slice, p.groups - g0), 0);
    const int wr = kWarps / p.wk, wrow = warp / p.wk, wkk = warp % p.wk;
    // shared memory: B fragments [slice][4 words][tokens][64], meta [slice][TOK], the warps' scales [kWarps][2][MATS][16 rows]
    // [kChunk], the warps' sums [kWarps][tile] (if they are to be added), and with a cluster this CTA's sums
    // [batch * wr][tile]
    uint8_t* frags = lsmem;
    float2* meta = reinterpret_cast<float2*>(lsmem + size_t(p.slice) * tokens * 256);
    float* scales = reinterpret_cast<float*>(meta + p.slice * TOK) + warp * (2 * MATS * 16 * kChunk);
    float* part = reinterpret_cast<float*>(meta + p.slice * TOK) + kWarps * (2 * MATS * 16 * kChunk);
    const bool direct = p.wk == 1 && cs > 1;   // a warp's sums are the CTA's
    float* hold = direct ? part : part + kWarps * kTile;

    // Earlier writes on the stream, the codes and scales among them, are visible here only behind this grid's own wait,
    // so nothing is read ahead of it, although stage_kernel reads no weights.
    pdl_wait();

    const int lg = lane >> 2, lt = lane & 3;
    const bool odd = lg & 1;
    // This warp's pairs of groups of the slice: wkk, wkk + wk, .. (the warps of a tile read along its rows together)
    const int all_pairs = (ng + 1) / 2, pairs = max((all_pairs - wkk + p.wk - 1) / p.wk, 0);
    const int padded = max((pairs + kPairs - 1) / kPairs, 1) * kPairs;   // whole turns, so that a slot's place is fixed
    const bool ragged = (ng & 1) && pairs > 0 && (all_pairs - 1) % p.wk == wkk;   // the last pair has one group
    auto first_row = [&](int it) { return ((int64_t(it) * p.clusters + cluster) * wr + wrow) * 16; };
    // The next load: tile step, pair there, and the lane's first code line (row lg rounded down to even,
    // group lg & 1) of each matrix; distances to its other lines.
    uint4 q[kPairs][MATS][4];
    int l_it = 0, l_pair = 0;
    const uint8_t* l_code[MATS];
    bool l_live = false;
    const int row_bytes = p.K / 2;
    const int to_next = row_bytes + (odd ? -64 : 64);   // the neighbouring row's line, the other group
    int to_8 = 0;                                       // rows 8 to 15, if the tile has them (else row lg again)
    auto enter = [&]() {
        const int64_t row = first_row(l_it);
        l_live = l_it < p.iters && row < p.N;
        if (!l_live) return;
        to_8 = row + 8 < p.N ? 8 * row_bytes : 0;
        const int64_t at = (row + (lg & ~1)) * row_bytes + (g0 + 2 * wkk + int(odd)) * 64 + lt * 16;
#pragma unroll
        for (int w = 0; w < MATS; ++w) l_code[w] = p.codes[w] + at;
    };
    auto load = [&](uint4 (&qd)[4], int mat, bool last) {
        if (l_live && l_pair < pairs) {
            const uint8_t *c = l_code[mat], *c1 = c + to_next;
            if (ragged && l_pair + 1 == pairs) {   // the second group's lanes read the first one again (their sums are dropped)
                if (odd) c -= 64;
                if (!odd) c1 -= 64;
            }
            qd[0] = __ldcs(reinterpret_cast<const uint4*>(c));
            qd[1] = __ldcs(reinterpret_cast<const uint4*>(c1));
            qd[2] = __ldcs(reinterpret_cast<const uint4*>(c + to_8));
            qd[3] = __ldcs(reinterpret_cast<const uint4*>(c1 + to_8));
            l_code[mat] += p.wk * 128;
        }
        if (mat == MATS - 1) {
            ++l_pair;
            if (last && l_pair == padded) {   // (only the last slot of a turn can end a tile)
                l_pair = 0;
                ++l_it;
                enter();
            }
        }
    };
    // Scales come in chunks of kChunk groups (a 32-byte sector a row) of the warp's tile, copied to shared memory one
    // chunk ahead: loaded per pair by the lanes that use them, they cost 16 requests where the codes take as
    // many, and a quarter of the time. One scale per row: one chunk a tile, of one column.
    const bool by_row = p.scale_groups == 1;
    const bool wide = (p.scale_groups & 1) == 0 && ((reinterpret_cast<uintptr_t>(p.scales[0]) |
                                                     reinterpret_cast<uintptr_t>(p.scales[MATS - 1])) & 7) == 0;
    int s_it = 0, s_at = 0, s_buf = 0;        // the next chunk: tile step, first of the warp's groups, buffer
    auto fetch_scales = [&]() {
        const int64_t row0 = first_row(s_it);
        if (s_it < p.iters && row0 < p.N && pairs > 0) {
            float* dst = scales + s_buf * (MATS * 16 * kChunk);
#pragma unroll
            for (int w = 0; w < MATS; ++w) {
                if (by_row) {
                    const int r = lane & 15;
                    if (lane < 16) copy_async<4>(dst + (w * 16 + r) * kChunk, p.scales[w] + min(row0 + r, int64_t(p.N) - 1));
                } else if (wide) {
#pragma unroll
                    for (int i = 0; i < 16 * kChunk / 64; ++i) {
                        const int at = 2 * (lane + 32 * i), r = at / kChunk, g = at % kChunk;
                        const int group = 2 * (wkk + (s_at + g) / 2 * p.wk) + (g & 1);
                        if (group < ng)
                            copy_async<8>(dst + w * 16 * kChunk + at,
                                          p.scales[w] + min(row0 + r, int64_t(p.N) - 1) * p.scale_groups + g0 + group);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16 * kChunk / 32; ++i) {
                        const int at = lane + 32 * i, r = at / kChunk, g = at % kChunk;
                        const int group = 2 * (wkk + (s_at + g) / 2 * p.wk) + (g & 1);
                        if (group < ng)
                            copy_async<4>(dst + w * 16 * kChunk + at,
                                          p.scales[w] + min(row0 + r, int64_t(p.N) - 1) * p.scale_groups + g0 + group);
                    }
                }
            }
        }
        s_buf ^= 1;
        s_at += kChunk;
        if (by_row || s_at >= 2 * pairs) {
            s_at = 0;
            ++s_it;
        }
    };
    uint4 raw[2];
    if (!p.staged) fetch_x(p, m0, ng * tokens, g0, ng, warp * 4, raw);
    enter();
#pragma unroll
    for (int d = 0; d < kPairs; ++d)
#pragma unroll
        for (int w = 0; w < MATS; ++w) load(q[d][w], w, d == kPairs - 1);
    fetch_scales();
    if (p.staged) {
        const uint8_t* src = staged_frags<TOK>(p, blockIdx.y) + size_t(g0) * tokens * 256;
        for (int i = threadIdx.x; i < ng * tokens * 16; i += kWarps * 32) copy16_async(frags + 16 * i, src + 16 * i);
        const float2* msrc = staged_meta<TOK>(p, blockIdx.y) + size_t(g0) * TOK;
        for (int i = threadIdx.x; i < ng * TOK / 2; i += kWarps * 32) copy16_async(meta + 2 * i, msrc + 2 * i);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        stage_x<FP4, TOK>(p, m0, tokens, g0, ng, warp, kWarps, raw, frags, meta);
    }
    pdl_trigger();
    __syncthreads();

    // the lane's B fragments: token bm of each eight (one that exists: what the spare columns compute is dropped)
    uint32_t frag0[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int bm = min(nt * 8 + lg, tokens - 1);
        frag0[nt] = uint32_t(2 * wkk * 4 * tokens + bm) * 64 + lt * 16;   // (from `frags`)
    }
    const uint32_t meta0 = uint32_t(p.slice) * tokens * 256 + uint32_t(2 * wkk * TOK + 2 * lt) * 8;
    float total[MATS][2][NT][4] = {};        // [matrix][group of the pair]
    int c_buf = 0;                           // the scales' buffer in use
    int held = 0;                            // tile steps whose sums wait for the cluster
    const uint32_t hold_addr = static_cast<uint32_t>(__cvta_generic_to_shared(hold));

    // one group of each matrix: rows' codes u[matrix][lg, lg + 8], their scales s
    auto group = [&](const uint32_t (&u)[MATS][2][4], const float (&s)[MATS][2], uint32_t fa, uint32_t ma, int half) {
        if constexpr (FP4) {
            float acc[MATS][NT][4] = {};
#pragma unroll
            for (int w4 = 0; w4 < 4; ++w4) {
                uint4 b[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    b[nt] = *reinterpret_cast<const uint4*>(lsmem + (frag0[nt] + fa + w4 * tokens * 64));
#pragma unroll
                for (int w = 0; w < MATS; ++w) {
                    uint32_t pa[4], pb[4];
                    decode_e2m1(u[w][0][w4], pa);
                    decode_e2m1(u[w][1][w4], pb);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_16816(acc[w][nt], pa[0], pb[0], pa[1], pb[1], b[nt].x, b[nt].y);
                        mma_16816(acc[w][nt], pa[2], pb[2], pa[3], pb[3], b[nt].z, b[nt].w);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 mm = *reinterpret_cast<const uint4*>(lsmem + (ma + nt * 64));   // two tokens' (0, scale)
#pragma unroll
                for (int w = 0; w < MATS; ++w)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float& t = total[w][half][nt][e];
                        t = fmaf(s[w][e >> 1] * __uint_as_float(e & 1 ? mm.w : mm.y), acc[w][nt][e], t);
                    }
            }
        } else {
            int hi[MATS][NT][4] = {}, lo[MATS][NT][4] = {};
#pragma unroll
            for (int w4 = 0; w4 < 4; ++w4) {
                uint4 b[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    b[nt] = *reinterpret_cast<const uint4*>(lsmem + (frag0[nt] + fa + w4 * tokens * 64));
#pragma unroll
                for (int w = 0; w < MATS; ++w) {
                    const uint32_t u0 = u[w][0][w4], u1 = u[w][1][w4];
                    const uint32_t a0 = (u0 & 0x0F0F0F0Fu) ^ 0x08080808u, a1 = (u1 & 0x0F0F0F0Fu) ^ 0x08080808u;
                    const uint32_t a2 = ((u0 >> 4) & 0x0F0F0F0Fu) ^ 0x08080808u;
                    const uint32_t a3 = ((u1 >> 4) & 0x0F0F0F0Fu) ^ 0x08080808u;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_u8s8(hi[w][nt], a0, a1, a2, a3, b[nt].x, b[nt].y);
                        mma_u8u8(lo[w][nt], a0, a1, a2, a3, b[nt].z, b[nt].w);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 mm = *reinterpret_cast<const uint4*>(lsmem + (ma + nt * 64));   // (15 sum(x), half the step)
#pragma unroll
                for (int w = 0; w < MATS; ++w)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // 2 (256 hi + lo) - 15 sum(x), below 2^28 in magnitude
                        const int v = int(uint32_t(512 * hi[w][nt][e] + 2 * lo[w][nt][e]) - (e & 1 ? mm.z : mm.x));
                        float& t = total[w][half][nt][e];
                        t = fmaf(s[w][e >> 1] * __uint_as_float(e & 1 ? mm.w : mm.y), __int2float_rn(v), t);
                    }
            }
        }
    };
#pragma unroll 1
    for (int it = 0; it < p.iters; ++it) {
        const int64_t row0 = first_row(it);
        const bool live = row0 < p.N;
        uint32_t frag_at = 0, meta_at = meta0;
        const float* c_scale = scales;
#pragma unroll 1
        for (int pair = 0; pair < padded; pair += kPairs) {
            if ((2 * pair) % kChunk == 0 && (pair == 0 || (!by_row && pair < pairs))) {
                // a new chunk of scales: wait for its copies, ask for the next one
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                c_scale = scales + c_buf * (MATS * 16 * kChunk);
                c_buf ^= 1;
                fetch_scales();
            }
#pragma unroll
            for (int d = 0; d < kPairs; ++d) {
                if (live && pair + d < pairs) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == 1 && ragged && pair + d + 1 == pairs) break;
                        // even lanes: rows lg from loads 0 and 2 in the first group, lg + 1 from 1 and 3 in the
                        // second; odd lanes the other way round
                        uint32_t u[MATS][2][4];
                        float sv[MATS][2];
#pragma unroll
                        for (int w = 0; w < MATS; ++w) {
                            const uint4 a = odd == (h != 0) ? q[d][w][0] : q[d][w][1];
                            const uint4 b = odd == (h != 0) ? q[d][w][2] : q[d][w][3];
                            u[w][0][0] = a.x; u[w][0][1] = a.y; u[w][0][2] = a.z; u[w][0][3] = a.w;
                            u[w][1][0] = b.x; u[w][1][1] = b.y; u[w][1][2] = b.z; u[w][1][3] = b.w;
                            const float* s = c_scale + (w * 16 + (lg ^ h)) * kChunk +
                                             (by_row ? 0 : (2 * (pair + d) + h) % kChunk);
                            sv[w][0] = s[0];
                            sv[w][1] = s[8 * kChunk];
                        }
                        group(u, sv, frag_at + h * tokens * 256, meta_at + h * TOK * 8, h);
                    }
                }
#pragma unroll
                for (int w = 0; w < MATS; ++w) load(q[d][w], w, d == kPairs - 1);
                frag_at += p.wk * tokens * 512;
                meta_at += p.wk * TOK * 16;
            }
        }
        // the tile's sums
        float* dst = (direct ? hold + (held * wr + wrow) * kTile : part + warp * kTile) + lg;
#pragma unroll
        for (int w = 0; w < MATS; ++w)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // the second group's sums belong to the neighbouring row
                    const float t = total[w][0][nt][e] + __shfl_xor_sync(0xFFFFFFFFu, total[w][1][nt][e], 4);
                    dst[(w * TOK + nt * 8 + 2 * lt + (e & 1)) * 16 + 8 * (e >> 1)] = t;
                    total[w][0][nt][e] = total[w][1][nt][e] = 0.0f;
                }
        // the tile's wk warps: all sums written, and below all read before the next tile's
        auto meet = [&]() {
            if (p.wk > 1)
                asm volatile("bar.sync %0, %1;" ::"r"(1 + wrow), "r"(32 * p.wk) : "memory");
            else
                __syncwarp();
        };
        if (!direct) {
            meet();
            const float* src = part + wrow * p.wk * kTile;
            for (int i = wkk * 32 + lane; i < 16 * tokens; i += 32 * p.wk) {
                float v[MATS] = {};
                for (int k = 0; k < p.wk; ++k)
#pragma unroll
                    for (int w = 0; w < MATS; ++w) v[w] += src[k * kTile + w * TOK * 16 + i];
                if (cs > 1) {
#pragma unroll
                    for (int w = 0; w < MATS; ++w) hold[(held * wr + wrow) * kTile + w * TOK * 16 + i] = v[w];
                } else if (row0 + (i & 15) < p.N) {
                    float out = v[0];
                    if constexpr (GATED) out = v[0] * gate_sigmoid<ACT>(v[0]) * v[1];
                    p.y[int64_t(m0 + (i >> 4)) * p.N + row0 + (i & 15)] = __float2bfloat16_rn(out);
                }
            }
            meet();
        }
        // in a cluster: a batch of tiles at a time, summed in rank order; the CTAs share the outputs
        if (cs > 1 && (++held == p.batch || it + 1 == p.iters)) {
            cluster_barrier();
            const int first = it + 1 - held, outs = held * wr * 16 * tokens;
            for (int i = int(rank) * kWarps * 32 + threadIdx.x; i < outs; i += int(cs) * kWarps * 32) {
                const int slot = i / (16 * tokens), at = i - slot * (16 * tokens);
                const int64_t row =
                    ((int64_t(first + slot / wr) * p.clusters + cluster) * wr + slot % wr) * 16 + (at & 15);
                if (row >= p.N) continue;
                float v[MATS] = {};
                for (uint32_t c = 0; c < cs; ++c) {
                    uint32_t base;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base) : "r"(hold_addr), "r"(c));
#pragma unroll
                    for (int w = 0; w < MATS; ++w) {
                        float f;
                        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                     : "=f"(f)
                                     : "r"(base + uint32_t(slot * kTile + w * TOK * 16 + at) * 4)
                                     : "memory");
                        v[w] += f;
                    }
                }
                float out = v[0];
                if constexpr (GATED) out = v[0] * gate_sigmoid<ACT>(v[0]) * v[1];
                p.y[int64_t(m0 + (at >> 4)) * p.N + row] = __float2bfloat16_rn(out);
            }
            // no sum is overwritten, and no CTA leaves, while another may still read them
            cluster_barrier();
            held = 0;
        }
    }
}

// Clusters of `cs` CTAs of a kernel that run at the same time on the current device (asked once per kernel, device
// and cs, at the shared memory in cfg).
int active_clusters(const void* kernel, const cudaLaunchConfig_t& cfg, int cs) {
    struct Entry {
        const void* kernel;
        int dev, cs, n;
    };
    constexpr int kSlots = 96;   // more than the kernels times the cluster sizes of one device; older entries give way
    static Entry cache[kSlots] = {};
    static int next = 0;
    static std::mutex mu;
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry& e : cache)
        if (e.kernel == kernel && e.dev == dev && e.cs == cs) return e.n;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = sm_count() / cs > 0 ? sm_count() / cs : 1;
    }
    cache[next] = {kernel, dev, cs, n};
    next = (next + 1) % kSlots;
    return n;
}

template <bool FP4, int NT, bool GATED, int ACT>
cudaError_t launch_one(const LowbitArgs& a, cudaStream_t stream) {
    constexpr int MATS = GATED ? 2 : 1, TOK = 8 * NT;
    constexpr size_t kTileBytes = MATS * TOK * 16 * 4;
    LowbitParams p;
    p.x = reinterpret_cast<const __nv_bfloat16*>(a.x);
    p.ld_x = a.ld_x;
    for (int w = 0; w < 2; ++w) {
        p.codes[w] = a.codes[w];
        p.scales[w] = a.scales[w];
    }
    p.y = reinterpret_cast<__nv_bfloat16*>(a.y);
    p.staged = static_cast<uint8_t*>(a.workspace);   // null below lowbit_workspace_bytes' limit
    p.M = (int)a.M; p.N = (int)a.N; p.K = (int)a.K; p.had = a.had;
    p.groups = (int)(a.K / kGroup);
    p.scale_groups = a.scale_groups;
    p.had_scale = a.had ? (float)(1.0 / sqrt((double)a.had)) : 1.0f;
    const int tokens = p.M < TOK ? p.M : TOK, token_tiles = (p.M + TOK - 1) / TOK;
    const int64_t tiles = (int64_t(p.N) + 15) / 16;
    // whole pairs of groups (blocks of 256 columns stay together); one CTA takes them all
    auto slice_of = [&](int c) { return c == 1 ? p.groups : ((p.groups + c - 1) / c + 1) / 2 * 2; };
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
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;

    // CTAs along K (cs) and warps along K (wk): the pair with the least work for the busiest warp, counted in
    // groups: its row tiles, each ceil(slice / wk) groups and a sum over the warps worth about three, and
    // each batch's sum over the cluster about four. Larger clusters leave SMs empty (their CTAs share a GPC), so the
    // clusters that run at once are asked of the runtime. Shared memory must hold the slice of x, the warps' sums and, in
    // a cluster, every tile's sums. With a warp sum worth 0, 1, 3, 6 and 12 groups: 1 x 44032 x 8192 73, 51, 51, 51 and 59 us,
    // gated 1 x 22016 x 8192 52, 52, 52, 56 and 69, gated 16 x 22016 x 8192 141, 92, 87, 87 and 87; with a cluster sum worth 0,
    // 4, 8 and 16 the last takes 92, 87, 87 and 87. Layers below 10 us differ by 0.2 at most in all of these.
    constexpr size_t kRoom = 226 * 1024;
    static_assert(kLowbitMaxK / kGroup / kMaxCluster * (TOK * 256 + TOK * 8) + kWarps * (2 * MATS * 16 * kChunk * 4) +
                          kWarps * kTileBytes + kTileBytes <= kRoom,
                  "the longest rows fit with the largest cluster and all warps along K");
    int cs = 0;
    int64_t best = 0, clusters = 0;
    size_t smem = 0;
    for (int c = 1; c <= kMaxCluster; c *= 2) {
        const int slice = slice_of(c);
        if (c > 1 && slice == slice_of(c / 2)) break;
        const size_t fixed = size_t(slice) * (tokens * 256 + TOK * 8) + kWarps * (2 * MATS * 16 * kChunk * 4);
        if (fixed > kRoom) continue;
        attr[1].val.clusterDim.x = c;
        cfg.gridDim = dim3((unsigned)c);
        cfg.dynamicSmemBytes = kRoom;
        int64_t wave = active_clusters((const void*)kernel, cfg, c) / token_tiles;
        if (wave < 1) wave = 1;
        for (int wk = 1; wk <= kWarps && (wk == 1 || 2 * wk <= slice + 1); wk *= 2) {
            const int side = kWarps / wk;
            const int64_t turns = (tiles + side - 1) / side;
            const int64_t iters = (turns + wave - 1) / wave;
            size_t need = fixed + (c > 1 && wk == 1 ? 0 : kWarps * kTileBytes);
            if (need > kRoom) continue;
            int64_t batch = iters;
            if (c > 1) {   // as many tiles at a time as shared memory holds sums of
                batch = int64_t((kRoom - need) / (side * kTileBytes));
                if (batch < 1) continue;
                if (batch > iters) batch = iters;
                need += size_t(batch) * side * kTileBytes;
            }
            const int64_t used = (turns + iters - 1) / iters;
            const int per_warp = ((slice + 1) / 2 + wk - 1) / wk;
            const int64_t cost = iters * (2 * per_warp + 3) + (c > 1 ? (iters + batch - 1) / batch * 4 : 0);
            if (cs == 0 || cost < best) {
                best = cost;
                cs = c;
                clusters = used;
                smem = need;
                p.wk = wk;
                p.slice = slice;
                p.iters = (int)iters;
                p.batch = (int)batch;
            }
        }
    }
    p.clusters = (int)clusters;
    if (p.staged) {
        const dim3 grid((unsigned)((p.groups * tokens + 15) / 16), (unsigned)token_tiles);
        const cudaError_t e = launch_pdl(stage_kernel<FP4, TOK>, grid, dim3(128), 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    cfg.gridDim = dim3((unsigned)(p.clusters * cs), (unsigned)token_tiles);
    cfg.dynamicSmemBytes = smem;
    attr[1].val.clusterDim.x = cs;
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

// x is transformed by a kernel of its own from this many (token, group) items on; below, every CTA transforms its slice.
// With the limit at 64, 128, 256 and 512 (replayed graphs of 24 calls): 4 x 5632 x 2048 6.9, 6.5, 6.5 and 6.5 us, 8 x 2048
// x 2048 6.2, 6.2, 7.1 and 7.1, 16 x 2048 x 2048 6.4, 6.5, 6.5 and 9.5, 4 x 2048 x 8192 7.7, 7.6, 7.7 and 10.6.
constexpr int64_t kStageItems = 128;

size_t lowbit_workspace_bytes(int64_t M, int64_t K) {
    const int64_t groups = K / kGroup;
    if (M * groups < kStageItems) return 0;
    return size_t(groups) * (size_t(M) * 256 + size_t(M + 15) / 16 * 16 * 8);
}

cudaError_t launch_lowbit(const LowbitArgs& a, cudaStream_t stream) {
    if (a.M == 0 || a.N == 0) return cudaSuccess;
    if (a.K == 0) return launch_zero_fill(a.y, nullptr, a.M * a.N, stream);
    return a.fp4 ? launch_grid<true>(a, stream) : launch_grid<false>(a, stream);
}

}  // namespace quest
