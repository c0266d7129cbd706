// The gate activation of the feed-forward block and the 8-bit checkpoint of a
// projection, shared by the block's kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "quest.h"

namespace quest {
namespace {

// act(a) = a s(a), s = sigmoid(z(a)): z = a (SiLU) or z = 2 sqrt(2/pi) (a + 0.044715 a^3)
// (the tanh form of GELU, since (1 + tanh(u)) / 2 = sigmoid(2 u)). exp and the quotient are
// the fast intrinsics. Their error grows with the argument, about 2 + 1.2 |z| units in the last place: a few 1e-7 for
// small |z|, up to 1.3e-5 (2^-16) for z near -87, where all of it reaches s, still 2^-8 of the bf16 outputs' rounding.
// The quotient is 0 for a divisor above 2^126, so s is 0 from z < -87.3 on, off by at most 2^-126; exp overflows
// to infinity for z < -88.7, where the quotient is 0 as it should be.
constexpr float kGeluZ = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

template <int ACT>
__device__ __forceinline__ float gate_sigmoid(float a) {
    const float z = ACT == QUEST_ACT_SILU ? a : kGeluZ * fmaf(kGeluC * a * a, a, a);
    return __fdividef(1.0f, 1.0f + __expf(-z));
}

// d/da [a s(a)] = s + a s (1 - s) z'(a), given s = s(a). Where s (1 - s) has rounded to zero the
// second term is zero, whatever z' is (it overflows for |a| > 1e19).
template <int ACT>
__device__ __forceinline__ float gate_slope(float a, float s) {
    const float p = s * (1.0f - s);
    if (ACT == QUEST_ACT_SILU) return fmaf(a, p, s);
    const float dz = kGeluZ * fmaf(3.0f * kGeluC * a, a, 1.0f);
    return p == 0.0f ? s : fmaf(a * p, dz, s);
}

// 8-bit checkpoint of a group of up to 128 consecutive columns of a row: Delta = max|v| / 128,
// q = floor(v / Delta), restored as (q + 1/2) Delta, the midrise form of the quantizer's codes. The quotient is
// v * inv with inv 1.5 2^-22 below 1 / Delta at most (ckpt_scale), so a value at k Delta, |k| <= 128, counts as below
// the boundary up to 1.5 2^-15 Delta above it; with the restored product's rounding, 2^-17 Delta, the error is at
// most (1/2 + 2^-14) Delta everywhere, the group's largest value included. Magnitudes are compared as
// bit patterns, so that a NaN wins and the whole group restores to NaN (an infinity: to infinities).
constexpr float kCkptMagic = 12582912.0f;   // 1.5 * 2^23: x + magic holds floor(x) in its low bits under rounding down

struct CkptScale {
    float delta;   // stored
    float inv;     // 1 / Delta, 2^-22 below it, so that |v| inv < 128 and no clamp is needed
};

__device__ __forceinline__ CkptScale ckpt_scale(uint32_t amax_bits) {
    const float amax = __uint_as_float(amax_bits);
    CkptScale r;
    // a group below 2^-100 is kept as zeros: 1 / Delta would overflow near the bottom of the range
    const bool tiny = amax < 7.888609052210118e-31f;
    r.delta = tiny ? 0.0f : amax * 0.0078125f;
    r.inv = tiny ? 0.0f : __frcp_rn(r.delta) * (1.0f - 2.384185791015625e-7f);
    return r;
}

// Four codes, little-endian in a word.
__device__ __forceinline__ uint32_t ckpt_pack4(float v0, float v1, float v2, float v3, float inv) {
    const uint32_t q0 = __float_as_uint(__fmaf_rd(v0, inv, kCkptMagic)), q1 = __float_as_uint(__fmaf_rd(v1, inv, kCkptMagic));
    const uint32_t q2 = __float_as_uint(__fmaf_rd(v2, inv, kCkptMagic)), q3 = __float_as_uint(__fmaf_rd(v3, inv, kCkptMagic));
    return __byte_perm(__byte_perm(q0, q1, 0x0040), __byte_perm(q2, q3, 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace
}  // namespace quest
