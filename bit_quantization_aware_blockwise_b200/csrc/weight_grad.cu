// Weight gradient of the quantized linear layer from the saved codes of its input,
// with the trust backward fused into the epilogue.
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

#include "tc_common.cuh"

namespace quest {
namespace {

// ---------------------------------------------------------------------------
//   G[n][k]  = sum_t gy[t][n] xh[t][k],  xh[t][k] = bf16((q[t][k] + 1/2) Delta[t][group of k])
//   gw[n][b] = H (mask[n][b] * G[n][b]) / sqrt(128)   per 128-column block b of a row
//
// Two launches. A streaming pass restores xh into the workspace (byte -> fp32 by a byte permute
// onto 2^15, minus the offset, times the token's step, rounded to bf16, as the quantizer's dequant is but for
// rare ties): 3 bytes moved per value. The product then runs at the tensor cores' rate. Restoring inside
// the product's mainloop instead repeats the work for every 256 rows of G: eight conversion warps
// beside the MMAs took 694 us at 16384 x 11264 x 2048 (541 with the conversion's arithmetic and stores
// taken out) where the pass costs 20 us and all of it 502 (single calls; 599-647 back to back, as the power cap settles).
//
// The reduction runs over the tokens, the outer dimension of both operands, so the MMA
// takes both transposed (MN-major): a stage row is one token's 64 columns (128 bytes,
// 128-byte swizzle), which is how gy [T, N] and xh [T, K] lie in memory. Nothing is transposed.
//
// CTA pairs, M = 256 rows of G, N = 256 columns, K = 16 tokens per MMA, 64 tokens per stage.
// Three warpgroups per CTA: one holds the TMA producer and (in the even CTA) the MMA issuer,
// two are epilogue teams, one per 128-column half; registers move to the teams (setmaxnreg).
//
// The tensor core adds to its fp32 accumulator by cutting, so a sum of T / 16 steps drifts by about
// T / 16 * 2^-26 of its value. An accumulator therefore holds at most one segment of the tokens;
// the teams add it to fp32 registers, rounding to nearest, while the MMAs fill the other one.
// Segments of 512 tokens keep an fp32 gradient within 6e-7 (2-norm; 4.3e-6 for 4096 tokens
// without them); a bf16 gradient is off by 1.7e-3 through its own rounding, and takes segments of 4096.
constexpr int kWThreads = 384;
constexpr int kTeamThreads = 128;
constexpr int kTokens = 64;                                // tokens per stage
constexpr int kSegF32 = 512 / kTokens, kSegBf16 = 4096 / kTokens;
constexpr uint32_t kWBox = kTokens * 128;                  // one 64-column box: 64 rows of 128 bytes
constexpr int kWStages = 6;
constexpr uint32_t kWStageA = 2 * kWBox, kWStageB = 2 * kWBox;
constexpr uint32_t kWChunk = BM * 64;                      // epilogue staging: 128 rows of 64 bytes, two a team
constexpr uint32_t kWSmemA = 0;
constexpr uint32_t kWSmemB = kWSmemA + kWStages * kWStageA;
constexpr uint32_t kWSmemC = kWSmemB + kWStages * kWStageB;
constexpr uint32_t kWSmemBar = kWSmemC + 4 * kWChunk;
constexpr uint32_t kWNumBars = 2 * kWStages + 4 + 1;
constexpr uint32_t kWSmemTmemSlot = kWSmemBar + kWNumBars * 8;
constexpr uint32_t kWSmemAbort = kWSmemTmemSlot + 4;
constexpr uint32_t kWSmemTotal = kWSmemAbort + 4 + 1024;
static_assert(kWSmemTotal <= 227 * 1024, "weight gradient shared memory");

// Registers per thread: 128 * (56 + 2 * 224) = 64512, what the block is launched with (384 * 168).
constexpr int kRegsIssue = 56, kRegsTeam = 224;
static_assert(128 * (kRegsIssue + 2 * kRegsTeam) <= kWThreads * 168, "register split");
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void team_bar(int id) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kTeamThreads) : "memory");
}
__device__ __forceinline__ bool team_any(int id, bool pred) {
    uint32_t out;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(out)
        : "r"((uint32_t)pred), "r"(id), "n"(kTeamThreads)
        : "memory");
    return out != 0;
}

constexpr uint32_t kIdescBf16Mn = (1u << 4)      // D: fp32
                                | (1u << 7)      // A: bf16
                                | (1u << 10)     // B: bf16
                                | (1u << 15)     // A transposed (MN-major)
                                | (1u << 16)     // B transposed (MN-major)
                                | (uint32_t(BN >> 3) << 17) | (uint32_t(256 >> 4) << 24);

// MN-major tile of 64-column boxes with 128-byte rows, one row per token, 128-byte
// swizzle: boxes kWBox apart along M / N, groups of 8 tokens 1024 bytes apart along K.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t addr) {
    uint64_t d = 0;
    d |= uint64_t((addr >> 4) & 0x3FFFu);
    d |= uint64_t(kWBox >> 4) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;                        // descriptor version (sm_100)
    d |= uint64_t(2) << 61;                        // layout: 128-byte swizzle
    return d;
}

__device__ __forceinline__ void tc_mma_bf16_mn_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                    uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(kIdescBf16Mn), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
}

struct WeightGradParams {
    const uint8_t* mask;        // trust mask bits of the weight [N, K / 8], or null (all kept)
    int T, N, K;
    int num_n, num_k;           // 256-row and 256-column tiles of G
    int splits, blocks_per_split, num_tb;   // token blocks of 64: in all, and per split
    int raw_rows;               // rows of one split's slice of the workspace
    int add;                    // fp32 output: added to what is there
};

enum { kOutBf16 = 0, kOutF32 = 1, kOutRaw = 2 };

// Unnormalised 128-point Walsh-Hadamard transform (Sylvester order) of one thread's registers.
__device__ __forceinline__ void fwht128(float2 (&w)[64]) {
#pragma unroll
    for (int j = 0; j < 64; ++j) w[j] = make_float2(w[j].x + w[j].y, w[j].x - w[j].y);
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) {
#pragma unroll
        for (int j = 0; j < 64; ++j) {
            if ((j & h) == 0) {
                const float2 a = w[j], b = w[j + h];
                w[j] = __fadd2_rn(a, b);
                w[j + h] = __ffma2_rn(b, make_float2(-1.0f, -1.0f), a);
            }
        }
    }
}

constexpr float kInvSqrt128 = 0.08838834764831845f;

// Four unsigned code bytes -> four bf16 values (two words).
__device__ __forceinline__ void convert4(uint32_t u, float2 neg_off, float2 step, uint32_t& lo, uint32_t& hi) {
    // 0x4700uu00 is 2^15 + uu
    const float2 a = make_float2(__uint_as_float(__byte_perm(u, 0x47000000u, 0x7404)),
                                 __uint_as_float(__byte_perm(u, 0x47000000u, 0x7414)));
    const float2 b = make_float2(__uint_as_float(__byte_perm(u, 0x47000000u, 0x7424)),
                                 __uint_as_float(__byte_perm(u, 0x47000000u, 0x7434)));
    const float2 va = __fmul2_rn(__fadd2_rn(a, neg_off), step), vb = __fmul2_rn(__fadd2_rn(b, neg_off), step);
    const __nv_bfloat162 ha = __floats2bfloat162_rn(va.x, va.y), hb = __floats2bfloat162_rn(vb.x, vb.y);
    lo = *reinterpret_cast<const uint32_t*>(&ha);
    hi = *reinterpret_cast<const uint32_t*>(&hb);
}

// The saved codes restored to bf16: xh [T, K], eight values (16 bytes out, 8 or 4 in) a thread and turn, neighbours'
// side by side, four turns' loads in flight. (Sixteen codes a thread left half-written sectors in each
// store instruction: 23 us where this takes 20.5 at 16384 x 2048 from 8 bits.)
struct RestoreParams {
    const uint8_t* codes;
    const float* scales;
    uint4* xh;
    int64_t chunks;             // T * per_row
    uint32_t per_row;           // groups of eight per token
    int scale_shift;            // group of eight in the row >> shift = group of 128 (31: one step per token)
    int64_t groups;
    float offset;               // code byte as unsigned -> value: (2^15 + u) - offset, times step * mul
    float mul;
    uint32_t flip;              // makes the stored two's complement fields unsigned
};

template <int CB>
__global__ void __launch_bounds__(256) restore_codes_kernel(const RestoreParams p) {
    pdl_wait();
    pdl_trigger();
    constexpr int kTurns = 4;
    const float2 neg_off = make_float2(-p.offset, -p.offset);
    const int64_t stride = int64_t(gridDim.x) * blockDim.x;
    for (int64_t i0 = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i0 < p.chunks; i0 += kTurns * stride) {
        uint32_t w[kTurns][2];
        float s[kTurns];
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int64_t i = i0 + k * stride;
            if (i < p.chunks) {
                // (below 2^32 values the row comes from a 32-bit division)
                const int64_t row = p.chunks >> 32 ? i / p.per_row : int64_t(uint32_t(i) / p.per_row);
                const uint32_t at = uint32_t(i - row * p.per_row);
                if constexpr (CB == 8) {
                    const uint2 q = __ldcs(reinterpret_cast<const uint2*>(p.codes) + i);
                    w[k][0] = q.x;
                    w[k][1] = q.y;
                } else {
                    w[k][0] = __ldcs(reinterpret_cast<const uint32_t*>(p.codes) + i);
                }
                s[k] = __ldg(p.scales + row * p.groups + (at >> p.scale_shift)) * p.mul;
            }
        }
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int64_t i = i0 + k * stride;
            if (i < p.chunks) {
                const float2 step = make_float2(s[k], s[k]);
                uint32_t o[4];
                if constexpr (CB == 8) {
                    convert4(w[k][0] ^ p.flip, neg_off, step, o[0], o[1]);
                    convert4(w[k][1] ^ p.flip, neg_off, step, o[2], o[3]);
                } else {
                    // low nibbles are the even elements, high nibbles the odd ones
                    const uint32_t u = w[k][0] ^ p.flip, ev = u & 0x0F0F0F0Fu, od = (u >> 4) & 0x0F0F0F0Fu;
                    convert4(__byte_perm(ev, od, 0x5140), neg_off, step, o[0], o[1]);
                    convert4(__byte_perm(ev, od, 0x7362), neg_off, step, o[2], o[3]);
                }
                p.xh[i] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

// OUT: kOutBf16 / kOutF32 finish the gradient; kOutRaw stores the plain sums of one token
// split for weight_grad_finish_kernel.
template <int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWThreads, 1)
weight_grad_kernel(const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ CUtensorMap map_o, const WeightGradParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    constexpr int kSeg = OUT == kOutBf16 ? kSegBf16 : kSegF32;
    const uint32_t bar_full = sbase + kWSmemBar;                 // [kWStages], used in the even CTA
    const uint32_t bar_empty = bar_full + 8 * kWStages;          // [kWStages]
    const uint32_t bar_tfull = bar_empty + 8 * kWStages;         // [2]
    const uint32_t bar_tempty = bar_tfull + 16;                  // [2], used in the even CTA
    const uint32_t bar_drain = bar_tempty + 16;                  // [1]
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kWSmemAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kWSmemTmemSlot);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool even = rank == 0;
    const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
    const int tiles = p.num_n * p.num_k;
    const int num_items = tiles * p.splits;   // split-major: the pairs in flight share a token range

    if (threadIdx.x == 0) {
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, 4);   // two teams in each CTA
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

    if (warp < 4) {
      regs_dec<kRegsIssue>();
      if (warp == 0) {
        // ------------------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            const uint32_t full_even = map_to_rank(bar_full, 0);
            uint32_t stage = 0, phase = 0;
            uint64_t issued = 0;
            bool ok = true;
            for (int item = pair; item < num_items && ok; item += num_pairs) {
                const int tile = item % tiles, split = item / tiles;
                const int n0 = (tile / p.num_k) * 256 + 128 * int(rank);
                const int k0 = (tile % p.num_k) * BN + 128 * int(rank);
                const int tb0 = split * p.blocks_per_split, tb1 = min(tb0 + p.blocks_per_split, p.num_tb);
                for (int tb = tb0; tb < tb1; ++tb) {
                    if (!mbar_wait(bar_empty + 8 * stage, phase ^ 1, abort_flag, kWaitLimitNs, kSuspendProducerNs)) {
                        ok = false;
                        break;
                    }
                    if (even) mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * (kWStageA + kWStageB));
                    const uint32_t fb = full_even + 8 * stage;
                    const uint32_t a_dst = sbase + kWSmemA + stage * kWStageA, b_dst = sbase + kWSmemB + stage * kWStageB;
                    tma_load_2d_pair(a_dst, &map_g, n0, tb * kTokens, fb);
                    tma_load_2d_pair(a_dst + kWBox, &map_g, n0 + 64, tb * kTokens, fb);
                    tma_load_2d_pair(b_dst, &map_x, k0, tb * kTokens, fb);
                    tma_load_2d_pair(b_dst + kWBox, &map_x, k0 + 64, tb * kTokens, fb);
                    ++issued;
                    if (++stage == kWStages) { stage = 0; phase ^= 1; }
                }
            }
            // giving up: no CTA may leave while a copy into its shared memory is in flight
            if (!ok && even) {
                const uint64_t n = issued < kWStages ? issued : kWStages;
                for (uint64_t i = issued - n; i < issued; ++i) {
                    const uint32_t st = uint32_t(i % kWStages), ph = uint32_t((i / kWStages) & 1);
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
            int local = 0;   // segments so far
            for (int item = pair; item < num_items && ok; item += num_pairs) {
                const int split = item / tiles;
                const int tb0 = split * p.blocks_per_split, tb1 = min(tb0 + p.blocks_per_split, p.num_tb);
                for (int seg = tb0; seg < tb1 && ok; seg += kSeg, ++local) {
                    const int seg_end = min(seg + kSeg, tb1);
                    const uint32_t buf = local & 1, bphase = (local >> 1) & 1;
                    if (!mbar_wait(bar_tempty + 8 * buf, bphase ^ 1, abort_flag, kWaitLimitNs, kSuspendMmaNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + buf * BN;
                    for (int tb = seg; tb < seg_end; ++tb) {
                        if (!mbar_wait(bar_full + 8 * stage, phase, abort_flag, kWaitLimitNs, kSuspendMmaNs)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t a_addr = sbase + kWSmemA + stage * kWStageA;
                        const uint32_t b_addr = sbase + kWSmemB + stage * kWStageB;
#pragma unroll
                        for (int kk = 0; kk < kTokens / 16; ++kk) {
                            tc_mma_bf16_mn_pair(d_tmem, smem_desc_mn128(a_addr + kk * 2048),
                                                smem_desc_mn128(b_addr + kk * 2048), tb != seg || kk != 0);
                        }
                        tc_commit_pair_mc(bar_empty + 8 * stage);
                        if (++stage == kWStages) { stage = 0; phase ^= 1; }
                    }
                    if (ok) tc_commit_pair_mc(bar_tfull + 8 * buf);
                }
            }
            tc_commit_pair(bar_drain);
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(bar_drain, 0) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
      }
    } else {
        // ------------------------------------------------------------ epilogue teams (warps 4..11, both CTAs)
        regs_inc<kRegsTeam>();
        const int team = (warp - 4) >> 2;      // 128-column half of the tile
        const int et = threadIdx.x - 32 * (4 + 4 * team), bar_id = 1 + team;
        const int quarter = warp & 3;
        const int row_in_tile = quarter * 32 + lane;
        const uint32_t lane_addr = uint32_t(quarter * 32) << 16;
        const uint32_t tempty_even = map_to_rank(bar_tempty, 0);
        const uint32_t staging = sbase + kWSmemC + team * 2 * kWChunk;
        int local = 0;
        int cbuf = 0;
        bool ok = true;
        for (int item = pair; item < num_items && ok; item += num_pairs) {
            const int tile = item % tiles, split = item / tiles;
            const int n0 = (tile / p.num_k) * 256 + 128 * int(rank), k0 = (tile % p.num_k) * BN + 128 * team;
            const int tb0 = split * p.blocks_per_split, tb1 = min(tb0 + p.blocks_per_split, p.num_tb);
            float2 w[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) w[i] = make_float2(0.0f, 0.0f);
#pragma unroll 1
            for (int seg = tb0; seg < tb1; seg += kSeg, ++local) {
                const uint32_t buf = local & 1, bphase = (local >> 1) & 1;
                const bool got = mbar_wait(bar_tfull + 8 * buf, bphase, abort_flag, kWaitLimitNs, kSuspendEpilogueNs);
                if (team_any(bar_id, !got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t t_acc = tmem_base + lane_addr + buf * BN + 128 * team;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t r[16];
                    QUEST_TMEM_LD16(t_acc + 16 * c, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[8 * c + i] = __fadd2_rn(w[8 * c + i], make_float2(__uint_as_float(r[2 * i]),
                                                                            __uint_as_float(r[2 * i + 1])));
                }
                tc_fence_before();
                team_bar(bar_id);
                if (et == 0) mbar_arrive_remote(tempty_even + 8 * buf);
            }
            if (!ok) break;
            if (n0 >= p.N || k0 >= p.K) continue;   // nothing of this half is stored (the same for the whole team)
            if constexpr (OUT != kOutRaw) {
                const int n = n0 + row_in_tile;
                if (p.mask != nullptr && n < p.N) {
                    const uint4 mb = *reinterpret_cast<const uint4*>(p.mask + int64_t(n) * (p.K / 8) + k0 / 8);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t bits = c == 0 ? mb.x : c == 1 ? mb.y : c == 2 ? mb.z : mb.w;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2& v = w[16 * c + i];
                            v.x = (bits >> (2 * i)) & 1u ? v.x : 0.0f;
                            v.y = (bits >> (2 * i + 1)) & 1u ? v.y : 0.0f;
                        }
                    }
                }
                fwht128(w);
            }
            constexpr int kChunks = OUT == kOutBf16 ? 4 : 8;   // of 64 bytes a row: 32 bf16 or 16 fp32 columns
            constexpr float kScale = OUT == kOutRaw ? 1.0f : kInvSqrt128;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const uint32_t stg = staging + cbuf * kWChunk + row_in_tile * 64;
                const uint32_t swz = (row_in_tile >> 1) & 3;
#pragma unroll
                for (int q16 = 0; q16 < 4; ++q16) {
                    uint32_t o[4];
                    if constexpr (OUT == kOutBf16) {
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const float2 v = w[16 * c + 4 * q16 + h];
                            const __nv_bfloat162 hb = __floats2bfloat162_rn(v.x * kScale, v.y * kScale);
                            o[h] = *reinterpret_cast<const uint32_t*>(&hb);
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float2 v = w[8 * c + 2 * q16 + h];
                            o[2 * h] = __float_as_uint(v.x * kScale);
                            o[2 * h + 1] = __float_as_uint(v.y * kScale);
                        }
                    }
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stg + ((q16 ^ swz) << 4)), "r"(o[0]),
                                 "r"(o[1]), "r"(o[2]), "r"(o[3])
                                 : "memory");
                }
                fence_proxy_async_smem();
                team_bar(bar_id);
                if (et == 0) {
                    const int col = k0 + c * (128 / kChunks);
                    const uint32_t src = staging + cbuf * kWChunk;
                    if (OUT == kOutRaw)
                        tma_store_2d(&map_o, src, col, split * p.raw_rows + n0);
                    else if (OUT == kOutF32 && p.add)
                        tma_reduce_add_2d(&map_o, src, col, n0);
                    else
                        tma_store_2d(&map_o, src, col, n0);
                    bulk_commit();
                    bulk_wait_read_le1();
                }
                team_bar(bar_id);
                cbuf ^= 1;
            }
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

// Sum of the token splits' plain sums in split order, mask, transform, store: a warp per
// 128-column block of a row, four columns a lane.
template <typename Out>
__global__ void __launch_bounds__(256) weight_grad_finish_kernel(const float4* __restrict__ part, const uint8_t* mask,
                                                                 Out* out, int64_t n_rows, int K, int splits,
                                                                 int64_t raw_rows, int add) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t kblocks = K / 128, total = n_rows * kblocks;
    for (int64_t i = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; i < total;
         i += (int64_t(gridDim.x) * blockDim.x) >> 5) {
        const int64_t n = i / kblocks, kb = i % kblocks;
        float4 v = part[(n * K + kb * 128) / 4 + lane];
        for (int s = 1; s < splits; ++s) {
            const float4 u = part[((s * raw_rows + n) * K + kb * 128) / 4 + lane];
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        if (mask) {
            const uint32_t bits = mask[n * (K / 8) + kb * 16 + (lane >> 1)] >> (4 * (lane & 1));
            if (!(bits & 1)) v.x = 0.0f;
            if (!(bits & 2)) v.y = 0.0f;
            if (!(bits & 4)) v.z = 0.0f;
            if (!(bits & 8)) v.w = 0.0f;
        }
        const float2 a = make_float2(v.x + v.y, v.x - v.y), b = make_float2(v.z + v.w, v.z - v.w);
        float t[4] = {a.x + b.x, a.y + b.y, a.x - b.x, a.y - b.y};
#pragma unroll
        for (int h = 1; h < 32; h <<= 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float o = __shfl_xor_sync(0xFFFFFFFFu, t[j], h);
                t[j] = lane & h ? o - t[j] : t[j] + o;
            }
        }
        Out* dst = out + n * K + kb * 128 + 4 * lane;
        if constexpr (sizeof(Out) == 4) {
            float4* d4 = reinterpret_cast<float4*>(dst);
            float4 r = make_float4(t[0] * kInvSqrt128, t[1] * kInvSqrt128, t[2] * kInvSqrt128, t[3] * kInvSqrt128);
            if (add) {
                const float4 o = *d4;
                r.x += o.x; r.y += o.y; r.z += o.z; r.w += o.w;
            }
            *d4 = r;
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(t[0] * kInvSqrt128, t[1] * kInvSqrt128);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(t[2] * kInvSqrt128, t[3] * kInvSqrt128);
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
    }
}

// Token splits: with fewer output tiles than CTA pairs, the tokens are cut so that the pairs left idle
// take part, in pieces of at least kMinBlocks blocks of 64 tokens (a piece costs its partial's round trip
// through the workspace, 256 KB a tile, and the finishing launch). 8192 x 512 x 512 takes 22.5 us so and 47 uncut,
// 3001 x 520 x 384 15.6 and 23; with pieces of at least 2, 4 and 16 blocks the latter takes 16.4, 16.4 and 18.5.
constexpr int kMinBlocks = 8;

struct SplitPlan {
    int splits, blocks_per_split, num_tb;
    int64_t raw_rows;
};

SplitPlan plan_splits(int64_t T, int64_t N, int64_t K) {
    SplitPlan s;
    s.num_tb = (int)((T + kTokens - 1) / kTokens);
    s.raw_rows = (N + 255) / 256 * 256;
    const int64_t tiles = ((N + 255) / 256) * ((K + BN - 1) / BN);
    const int64_t pairs = sm_count() / 2;
    int64_t want = tiles >= pairs || tiles == 0 ? 1 : pairs / tiles;
    const int64_t most = s.num_tb / kMinBlocks > 1 ? s.num_tb / kMinBlocks : 1;
    if (want > most) want = most;
    s.blocks_per_split = s.num_tb > 0 ? (int)((s.num_tb + want - 1) / want) : 1;
    s.splits = s.num_tb > 0 ? (s.num_tb + s.blocks_per_split - 1) / s.blocks_per_split : 1;
    return s;
}

// The workspace: xh [T, K] bf16, then (with token splits) the splits' sums [splits, raw_rows, K] fp32.
int64_t xh_bytes(int64_t T, int64_t K) { return (T * K * 2 + 255) / 256 * 256; }

template <int CB>
cudaError_t launch_restore(const WeightGradArgs& a, cudaStream_t stream) {
    RestoreParams p;
    p.codes = a.codes;
    p.scales = a.scales;
    p.xh = static_cast<uint4*>(a.workspace);
    p.per_row = (uint32_t)(a.K / 8);
    p.chunks = a.T * int64_t(p.per_row);
    p.scale_shift = a.groups == 1 ? 31 : 4;
    p.groups = a.groups;
    p.offset = 32768.0f + a.offset;
    p.mul = a.mul;
    p.flip = CB == 8 ? 0x80808080u : 0x88888888u;
    const int64_t blocks = (p.chunks + 255) / 256;
    const int64_t most = int64_t(sm_count()) * max_ctas_per_sm((const void*)restore_codes_kernel<CB>, 256, 0);
    return launch_pdl(restore_codes_kernel<CB>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, stream, p);
}

template <int OUT>
cudaError_t launch_main(const WeightGradArgs& a, const SplitPlan& plan, cudaStream_t stream) {
    CUtensorMap mg, mx, mo;
    void* dst = OUT == kOutRaw ? static_cast<char*>(a.workspace) + xh_bytes(a.T, a.K) : a.out;
    const uint64_t rows = OUT == kOutRaw ? uint64_t(plan.splits) * plan.raw_rows : uint64_t(a.N);
    const bool bf = OUT == kOutBf16;
    if (!make_map_2d(&mg, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.gy, a.N, a.T, a.ld_gy * 2, 64, kTokens,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.workspace, a.K, a.T, a.K * 2, 64, kTokens,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_2d(&mo, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dst, a.K, rows,
                     a.K * (bf ? 2 : 4), bf ? 32 : 16, 128, CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    WeightGradParams p;
    p.mask = a.mask;
    p.T = (int)a.T; p.N = (int)a.N; p.K = (int)a.K;
    p.num_n = (int)((a.N + 255) / 256);
    p.num_k = (int)((a.K + BN - 1) / BN);
    p.splits = plan.splits;
    p.blocks_per_split = plan.blocks_per_split;
    p.num_tb = plan.num_tb;
    p.raw_rows = (int)plan.raw_rows;
    p.add = a.accumulate;
    static thread_local int attr_dev = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (attr_dev != dev) {
        cudaError_t e = cudaFuncSetAttribute(weight_grad_kernel<OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kWSmemTotal);
        if (e != cudaSuccess) return e;
        attr_dev = dev;
    }
    const int64_t items = int64_t(p.num_n) * p.num_k * p.splits;
    const int pairs = pair_clusters(dev, (const void*)weight_grad_kernel<OUT>, kWThreads, kWSmemTotal);
    const int grid_pairs = items < pairs ? (int)items : pairs;
    return launch_pdl(weight_grad_kernel<OUT>, dim3(2 * grid_pairs), dim3(kWThreads), kWSmemTotal, stream, mg, mx,
                      mo, p);
}

cudaError_t launch_product(const WeightGradArgs& a, const SplitPlan& plan, cudaStream_t stream) {
    if (plan.splits == 1) return a.out_fp32 ? launch_main<kOutF32>(a, plan, stream) : launch_main<kOutBf16>(a, plan, stream);
    cudaError_t e = launch_main<kOutRaw>(a, plan, stream);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (a.N * (a.K / 128) + 7) / 8;
    const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384));
    const float4* part =
        reinterpret_cast<const float4*>(static_cast<const char*>(a.workspace) + xh_bytes(a.T, a.K));
    if (a.out_fp32)
        return launch_pdl(weight_grad_finish_kernel<float>, grid, dim3(256), 0, stream, part, a.mask,
                          static_cast<float*>(a.out), a.N, (int)a.K, plan.splits, plan.raw_rows, a.accumulate);
    return launch_pdl(weight_grad_finish_kernel<uint16_t>, grid, dim3(256), 0, stream, part, a.mask,
                      static_cast<uint16_t*>(a.out), a.N, (int)a.K, plan.splits, plan.raw_rows, 0);
}

}  // namespace

size_t weight_grad_workspace_bytes(int64_t T, int64_t N, int64_t K) {
    if (T == 0 || N == 0 || K == 0) return 0;
    const SplitPlan s = plan_splits(T, N, K);
    return size_t(xh_bytes(T, K)) + (s.splits == 1 ? 0 : size_t(s.splits) * size_t(s.raw_rows) * size_t(K) * 4);
}

cudaError_t launch_weight_grad(const WeightGradArgs& a, cudaStream_t stream) {
    if (a.N == 0 || a.K == 0) return cudaSuccess;
    if (a.T == 0) {   // the empty sum: zero, or nothing to add
        if (a.out_fp32 && a.accumulate) return cudaSuccess;
        const int64_t halves = a.N * a.K * (a.out_fp32 ? 2 : 1);
        return launch_zero_fill(static_cast<uint16_t*>(a.out), nullptr, halves, stream);
    }
    const SplitPlan plan = plan_splits(a.T, a.N, a.K);
    const cudaError_t e = a.code_bits == 8 ? launch_restore<8>(a, stream) : launch_restore<4>(a, stream);
    return e != cudaSuccess ? e : launch_product(a, plan, stream);
}

int read_and_clear_weight_grad_status(cudaStream_t stream, cudaError_t* err) {
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
