// rope.cuh -- the position rotation's angles, shared by the kernels that turn heads.
#pragma once

#include "fkv_common.cuh"

namespace fkv {

constexpr int kRopeMaxAxes = 8;

// cos and sin of pos * f.  The angle is formed in turns, pos * (f / 2 pi), with
// 1 / (2 pi) and the products in two fp32 words: pos is split into two exact
// 16-bit parts, each product's rounding error comes from one fma, and whole
// turns leave before sin and cos see the rest.  With |pos * f| < 2^31 the angle
// is off by less than 2^-18 of a turn; for |pos * f| < 2^20 by about 2^-23.
__device__ __forceinline__ float2 cos_sin_of(int32_t pos, float f) {
    const float inv_hi = 0.15915494f;                          // RN(1 / (2 pi))
    const float inv_lo = 6.4206382e-09f;                       // 1 / (2 pi) - inv_hi
    const float ch = f * inv_hi;
    const float cl = fmaf(f, inv_lo, fmaf(f, inv_hi, -ch));
    const int32_t lo16 = pos & 0xFFFF;
    const float a = static_cast<float>(pos - lo16), b = static_cast<float>(lo16);
    const float ha = a * ch, hb = b * ch;
    float ea = fmaf(a, cl, fmaf(a, ch, -ha));
    const float eb = fmaf(b, cl, fmaf(b, ch, -hb));
    ea -= rintf(ea);                                           // |ha| past 2^24 leaves whole turns here
    const float r = ((ha - rintf(ha)) + (hb - rintf(hb))) + (ea + eb);
    float s, c;
    sincospif(2.f * r, &s, &c);
    return make_float2(c, s);
}

__device__ __forceinline__ float2 bf16x2_to_f32(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

}  // namespace fkv
