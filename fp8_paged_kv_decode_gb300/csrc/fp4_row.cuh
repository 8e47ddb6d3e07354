// fp4_row.cuh -- the 4-bit cache's token row and its conversions.
//
// One (token, KV head) row is FKV_FP4_ROW_BYTES = 72 bytes: 64 bytes of e2m1
// codes (byte j holds dim 2j in its low nibble and dim 2j + 1 in its high one)
// and then 8 e4m3 scales, one per block of 16 dims.  With g the KV head's fp32
// scale, a value is e2m1(code) * e4m3(scale) * g.  Codes and scales of a row
// lie together so that one contiguous copy brings any run of a page's rows,
// and a new token is one 72-byte write.
#pragma once

#include "fkv_common.cuh"

namespace fkv {

constexpr int kFp4Codes = 64;            // code bytes of a row; the scales follow
constexpr int kFp4Row = FKV_FP4_ROW_BYTES;
static_assert(kFp4Row == kFp4Codes + 8, "64 code bytes and 8 scales");

// The 8 e2m1 codes of a word (low nibble first) as four f16 pairs.  Exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&f)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(w));
}

// Two fp32 values to two e2m1 codes in a byte (`lo` in the low nibble), nearest
// with ties to the even code, magnitudes above 6 (and infinities) to 6.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float hi, float lo) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
        "cvt.u32.u8 %0, b;\n\t}"
        : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// One scale byte as an f16 pair (s, s).
__device__ __forceinline__ uint32_t e4m3_to_f16_pair(uint32_t byte) {
    return e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(byte, 0u, 0x4400u)));
}

// A lane's share of a K row in shared memory: the codes of scale blocks t and
// 4 + t (dims 16t .. 16t + 15 and 64 + 16t ..) and the blocks' scales as pairs.
__device__ __forceinline__ void ld_fp4_row(uint32_t row, int t, uint32_t (&w)[4], uint32_t (&s)[2]) {
    const uint2 a = ld_shared_v2(row + 8 * t), b = ld_shared_v2(row + 32 + 8 * t);
    const uint2 sc = ld_shared_v2(row + kFp4Codes);
    w[0] = a.x;
    w[1] = a.y;
    w[2] = b.x;
    w[3] = b.y;
    const uint32_t two = prmt(sc.x, sc.y, 0x4400u + 0x1111u * t);          // bytes t, t, 4 + t, 4 + t
    s[0] = e4m3x2_to_f16x2(static_cast<uint16_t>(two & 0xFFFFu));
    s[1] = e4m3x2_to_f16x2(static_cast<uint16_t>(two >> 16));
}

// A lane's share of a V row: the 16 values of scale block g as f16 pairs
// (code * scale, exact).
__device__ __forceinline__ void ld_fp4_block(uint32_t row, int g, uint32_t (&x)[8]) {
    const uint2 c = ld_shared_v2(row + 8 * g);
    const uint32_t s = e4m3_to_f16_pair(ld_shared_u8(row + kFp4Codes + g));
    uint32_t f[4];
    e2m1x8_to_f16(c.x, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = mul_f16x2(f[j], s);
    e2m1x8_to_f16(c.y, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[4 + j] = mul_f16x2(f[j], s);
}

}  // namespace fkv
