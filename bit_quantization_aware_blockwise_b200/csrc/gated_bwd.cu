// Gated feed-forward block, backward of the activation and the product from the 8-bit
// checkpoint that quest_gated_linear kept.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gated_act.cuh"
#include "quest_internal.h"

namespace quest {
namespace {

// With a, b restored from their codes, a = (q_a + 1/2) Delta_a and so on, s = sigmoid(z(a)):
//   grad_a = grad_h b (s + a s (1 - s) z'(a)),  grad_b = grad_h a s,  h = a s b (optional)
// An elementwise pass bound by memory: per element it reads 2 bytes of grad_h and 2 code bytes (and
// 8 bytes of steps per 128) and writes 4 (6 with h). A thread owns 8 columns of a row, so that
// grad_h and each output are one 16-byte access and the codes 8-byte ones; a group's step is shared by
// 16 neighbouring threads.
template <int ACT, bool H>
__global__ void __launch_bounds__(256) gated_bwd_kernel(const uint4* __restrict__ gh, const uint2* __restrict__ codes,
                                                        const float* __restrict__ scales, uint4* __restrict__ grad,
                                                        uint4* __restrict__ h, int64_t n, int w, int groups) {
    pdl_wait();
    pdl_trigger();
    // row and 8-column slot of the thread, carried along instead of divided anew
    const int64_t step = int64_t(gridDim.x) * blockDim.x;
    const int64_t first = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    int64_t row = first / w;
    int col = int(first - row * w);
    const int64_t row_step = step / w;
    const int col_step = int(step - row_step * w);
    for (int64_t i = first; i < n; i += step) {
        const uint4 g4 = __ldcs(gh + i);
        const uint2 qa = __ldcs(codes + row * (2 * int64_t(w)) + col);
        const uint2 qb = __ldcs(codes + row * (2 * int64_t(w)) + w + col);
        const float* sc = scales + row * (2 * int64_t(groups)) + (col >> 4);
        const float da = __ldg(sc), db = __ldg(sc + groups);
        uint32_t oa[4], ob[4], oh[4];
        const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float va[2], vb[2], vh[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = 2 * j + e, sh = 8 * (k & 3);
                const int ca = int(int8_t((k < 4 ? qa.x : qa.y) >> sh)), cb = int(int8_t((k < 4 ? qb.x : qb.y) >> sh));
                const float a = (float(ca) + 0.5f) * da, b = (float(cb) + 0.5f) * db;
                const float g = __uint_as_float(e ? gw[j] & 0xFFFF0000u : gw[j] << 16);
                const float s = gate_sigmoid<ACT>(a);
                va[e] = g * b * gate_slope<ACT>(a, s);
                vb[e] = g * a * s;
                vh[e] = a * s * b;
            }
            oa[j] = pack_bf16(va[0], va[1]);
            ob[j] = pack_bf16(vb[0], vb[1]);
            oh[j] = pack_bf16(vh[0], vh[1]);
        }
        uint4* out = grad + row * (2 * int64_t(w)) + col;
        __stcs(out, make_uint4(oa[0], oa[1], oa[2], oa[3]));
        __stcs(out + w, make_uint4(ob[0], ob[1], ob[2], ob[3]));
        if (H) __stcs(h + i, make_uint4(oh[0], oh[1], oh[2], oh[3]));
        row += row_step;
        col += col_step;
        if (col >= w) {
            col -= w;
            ++row;
        }
    }
}

template <int ACT, bool H>
cudaError_t launch_bwd(const GatedBwdArgs& a, cudaStream_t stream) {
    const int w = (int)(a.F / 8);
    const int64_t n = a.M * w;
    const int64_t blocks = (n + 255) / 256;
    const int64_t most = int64_t(sm_count()) * max_ctas_per_sm((const void*)gated_bwd_kernel<ACT, H>, 256, 0);
    return launch_pdl(gated_bwd_kernel<ACT, H>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, stream,
                      reinterpret_cast<const uint4*>(a.gh), reinterpret_cast<const uint2*>(a.codes), a.scales,
                      reinterpret_cast<uint4*>(a.grad), reinterpret_cast<uint4*>(a.h), n, w, (int)((a.F + 127) / 128));
}

}  // namespace

cudaError_t launch_gated_bwd(const GatedBwdArgs& a, cudaStream_t stream) {
    if (a.M == 0 || a.F == 0) return cudaSuccess;
    if (a.act == QUEST_ACT_SILU)
        return a.h ? launch_bwd<QUEST_ACT_SILU, true>(a, stream) : launch_bwd<QUEST_ACT_SILU, false>(a, stream);
    return a.h ? launch_bwd<QUEST_ACT_GELU_TANH, true>(a, stream) : launch_bwd<QUEST_ACT_GELU_TANH, false>(a, stream);
}

}  // namespace quest
