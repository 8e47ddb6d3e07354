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

// Two fp32 lanes in one register pair.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(__float_as_uint(x)), "r"(__float_as_uint(y)));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    uint32_t x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(v));
    return make_float2(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// One scale byte as an f16 pair (s, s).
__device__ __forceinline__ uint32_t e4m3_to_f16_pair(uint32_t byte) {
    return e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(byte, 0u, 0x4400u)));
}

// f times the low (0) or high (1) half of a pair of scales.
__device__ __forceinline__ uint32_t mul_f16_half(uint32_t f, uint32_t pair, int half) {
    const __half2 s = *reinterpret_cast<const __half2 *>(&pair);
    const __half2 d = __hmul2(*reinterpret_cast<const __half2 *>(&f), half ? __high2half2(s) : __low2half2(s));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// The scales of blocks t and 4 + t of a row in shared memory, as an f16 pair.
__device__ __forceinline__ uint32_t ld_fp4_scales(uint32_t row, int t) {
    const uint2 sc = ld_shared_v2(row + kFp4Codes);
    return e4m3x2_to_f16x2(static_cast<uint16_t>(prmt(sc.x, sc.y, 0x40u + 0x11u * t)));
}

// A lane's share of two V rows in shared memory: the codes of scale block g and
// the two rows' scales of it as an f16 pair.
struct Fp4Pair {
    uint2 c0, c1;
    uint32_t s;
};
__device__ __forceinline__ Fp4Pair ld_fp4_pair(uint32_t row0, uint32_t row1, int g) {
    Fp4Pair v;
    v.c0 = ld_shared_v2(row0 + 8 * g);
    v.c1 = ld_shared_v2(row1 + 8 * g);
    const uint32_t b0 = ld_shared_u8(row0 + kFp4Codes + g), b1 = ld_shared_u8(row1 + kFp4Codes + g);
    v.s = e4m3x2_to_f16x2(static_cast<uint16_t>(b0 | (b1 << 8)));
    return v;
}

// The values of dims 8w .. 8w + 7 of the block as f16 pairs (first row, second
// row).  The rows' nibbles are interleaved first, two operations for four
// dims, so that a converted byte is one dim of both rows; converting each row
// and then regrouping halves costs four.
__device__ __forceinline__ void fp4_pairs(const Fp4Pair &v, int w, uint32_t (&x)[8]) {
    const uint32_t a = w ? v.c0.y : v.c0.x, b = w ? v.c1.y : v.c1.x;
    const uint32_t even = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
    const uint32_t odd = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
    uint32_t e[4], o[4];
    e2m1x8_to_f16(even, e);
    e2m1x8_to_f16(odd, o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = mul_f16x2(e[j], v.s);
        x[2 * j + 1] = mul_f16x2(o[j], v.s);
    }
}

}  // namespace fkv
