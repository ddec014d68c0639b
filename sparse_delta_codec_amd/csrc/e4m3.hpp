// e4m3.hpp -- rows of E4M3 codes with a scale for each 128 columns: the rule that
// the norm, the group quantiser and their tests share, and silu.
//
// For a group with amax = max |x|:  s = fl32(amax / 448), or 1 where amax is below
// 2^-96 (its codes are then zeros of x's sign);  code = E4M3(fl32(x / s)), to
// nearest, ties to even.  So it is fp8_block_quant's rule but for its lower end:
// there a block's values are BF16 and amax / 448 is never zero, here they are
// float32 and amax / 448 would have few bits left below 2^-117.
#pragma once

#include "device.hpp"

namespace pulse {

constexpr int QG = 128;  // columns of a group

// the largest of the 16 lanes of a DPP row, in all of them
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    uint32_t o;
    o = dpp_mov<0x128, 0xf, 0xf>(0u, v); v = o > v ? o : v;  // row_ror:8, 4, 2, 1
    o = dpp_mov<0x124, 0xf, 0xf>(0u, v); v = o > v ? o : v;
    o = dpp_mov<0x122, 0xf, 0xf>(0u, v); v = o > v ? o : v;
    o = dpp_mov<0x121, 0xf, 0xf>(0u, v); v = o > v ? o : v;
    return v;
}

// The codes of eight columns of a group that 16 lanes share; the group's scale in *scale.
// The quotient without a division per element: with y = fl32(1 / s), q0 = fl32(x y) and
// the remainder r = x - s q0 of an FMA, fl32(q0 + r y) is the correctly rounded quotient
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) while nothing underflows, which the factor 2^40 on both sees to.
// A group that holds an infinity or a NaN has that in its scale (magnitudes are compared
// as integers, where a NaN is the largest), and no code of it stands for a number.
__device__ __forceinline__ u32x2 group_codes(const float (&x)[8], float *scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(x[i]) & 0x7FFFFFFFu;
        m = a > m ? a : m;
    }
    const float amax = __uint_as_float(row16_max(m));
    const float s = amax < 1.2621774483536188887e-29f ? 1.0f : amax / 448.0f;  // 2^-96; IEEE division
    const bool up = s < 1.152921504606846976e18f;                             // 2^60
    const float f = up ? 1099511627776.0f : 1.0f, ss = s * f;                 // 2^40
    const float y = 1.0f / ss;                                                // IEEE division
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float xs = x[i] * f, q0 = xs * y;
        q[i] = __builtin_fmaf(__builtin_fmaf(-q0, ss, xs), y, q0);
        if (q0 == 0.0f) q[i] = q0;  // a zero keeps its sign
    }
    u32x2 c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
        c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], v, true);
    }
    *scale = s;
    return c;
}

// g / (1 + e^-g) in float32, off by a few units of 2^-24: the exponential as 2^t 2^d with t the
// rounded product and d what its rounding left out (up to 2^-18 at |g| = 80).  Gates below -44.4 have
// 2^-64 of the exponential, beside which 1 is nothing, and give that factor back to the quotient:
// the exponential itself passes float32's range at -88.7, and its reciprocal is below the normal
// numbers, where the instruction gives zero, from -87.3 on, while the quotient is one down to -91.8.
// (FAR = false: for gates from kFarGate on, without that part.)
constexpr float kFarGate = -44.0f;

template <bool FAR = true>
__device__ __forceinline__ float silu(float g) {
    constexpr float kLog2e = 1.44269502162933349609375f, kRest = 1.925963033500011079e-8f, kLn2 = 0.693147182464599609375f;
    const float t = g * -kLog2e;
    const float d = __builtin_fmaf(g, -kRest, __builtin_fmaf(g, -kLog2e, -t));
    const bool far = FAR && t > 64.0f;
    const float p = __builtin_amdgcn_exp2f(far ? t - 64.0f : t);  // (the difference is exact below 192)
    // beyond, e^-g is nothing beside 1 or the quotient is zero, and d may be inf - inf
    const float e = fabsf(t) < 192.0f ? __builtin_fmaf(p, d * kLn2, p) : p;
    const float q = g * __builtin_amdgcn_rcpf(far ? e : 1.0f + e);
    return far ? q * 5.42101086242752217e-20f : q;  // 2^-64
}

// eight BF16 of 16 bytes as float32
__device__ __forceinline__ void widen8(const u32x4 &v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ u32x4 narrow8(const float (&x)[8]) {
    return u32x4{cast_pair(x[0], x[1]), cast_pair(x[2], x[3]), cast_pair(x[4], x[5]), cast_pair(x[6], x[7])};
}

}  // namespace pulse
