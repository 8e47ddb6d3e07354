// kv_append_rope.cu -- RMS norm and position rotation of a step's heads, with the
// keys and values going into the cache in the same pass.
//
//   y = x rsqrt(mean(x^2) + eps) w;  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
// with t = position * inv_freq per pair, for the query heads (written as bf16)
// and the key heads (quantised from their fp32 values, rounded once, and put into
// their slots); the value heads are quantised as they are.  Each row is read and
// written once: what a separate rotation writes of the keys and the append reads
// again, 512 bytes a (token, KV head), and one launch are saved.
//
// A warp serves one token, or part of its heads when there are few tokens; 16
// lanes take a head row, lane l the elements 8l .. 8l + 7 in one 16-byte load.  The
// other half of a pair is in the same lane where pairs are neighbours and rotary_dim
// / 16 lanes away otherwise, four shuffles of packed words.  With the lane's eight
// elements side by side a row's codes are one 8-byte store per lane (FP8), its scale
// blocks two lanes each (FP4), and no lane holds two rows' worth of layouts.  The
// weights go into the rotation's coefficients once per token:
//   own' = rs (own (w_own cos) + other (-+ w_other sin))
#include <cmath>

#include "fp4_row.cuh"
#include "rope.cuh"

namespace fkv {

constexpr int kArBlock = 128;
constexpr int kArUnroll = 4;                   // rows a half-warp has in flight
constexpr int kArBatch = 2 * kArUnroll;        // rows of a warp's batch

struct AppendRopeParams {
    const uint16_t *q, *k, *v;                 // bf16
    uint16_t *q_out;
    int64_t qs, ks, vs, qos;                   // token strides in elements
    const uint4 *q_weight, *k_weight;
    const int32_t *positions;
    const float *inv_freq;
    const uint8_t *axis_map;
    const int64_t *slots;
    const float *k_scale, *v_scale;
    uint8_t *k_cache, *v_cache;
    uint32_t *err;
    uint64_t total_slots;                      // pages x page_size
    int32_t n_tokens, hq, hkv, heads, parts, rows_per_warp, n_axes, half;
    uint32_t page_size;
    int32_t page_shift;                        // log2 of the page size, -1 if it is not a power of two
    float eps, rot_scale;
};

// The quotients x / b of two fp32 lanes, from b's correctly rounded reciprocal and one
// remainder correction (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990): the IEEE quotient for every bf16 x (the append's
// values), within an ulp of it for any other (a rotated key, itself rounded).
// For b in [2^-30, 2^30] and |x| <= 2^64; nb = (-b, -b), yy = (1/b, 1/b).
__device__ __forceinline__ float2 quotient2(float x, float y, uint64_t nb, uint64_t yy) {
    const uint64_t a = pack2(x, y), q0 = mul2(a, yy);
    uint64_t r, q;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(q0), "l"(nb), "l"(a));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(r), "l"(yy), "l"(q0));
    return unpack2(q);
}
__device__ __forceinline__ bool quotient2_scale(float b) { return b >= 0x1p-30f && b <= 0x1p30f; }   // false for NaN too
constexpr uint32_t kQuotient2Max = 0x5F800000u;                // bits of 2^64

// A KV head's scale, as the encoders want it.
struct HeadScale {
    float g, g6, y6;                                           // the scale, fl32(6 g) and its reciprocal
    uint64_t nb, yy;                                           // (-g, -g) and (1/g, 1/g)
};
template <int kKv>
__device__ __forceinline__ HeadScale head_scale(const float *scales, int h) {
    HeadScale s{};
    if (kKv == FKV_KV_BF16) return s;
    s.g = __ldg(scales + h);
    if (kKv == FKV_KV_FP8_E4M3) {
        const float y = __frcp_rn(s.g);
        s.nb = pack2(-s.g, -s.g);
        s.yy = pack2(y, y);
    } else {
        s.g6 = __fmul_rn(6.f, s.g);
        s.y6 = __frcp_rn(s.g6);
    }
    return s;
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// One lane's 8 elements of a row, encoded and stored at the row's place (nullptr: a
// row that is not written; its lanes still take part in the shuffles).  `half_mask`:
// the 16 lanes of the row.
template <int kKv>
__device__ __forceinline__ void store_cached(uint8_t *row, int lane, unsigned half_mask, const float (&x)[8], const HeadScale &hs) {
    if (kKv == FKV_KV_BF16) {
        if (row) __stcs(reinterpret_cast<uint4 *>(row) + lane, pack_bf16x8(x));
        return;
    }
    uint32_t big = 0;                                          // a NaN's bits are above every other value's
#pragma unroll
    for (int e = 0; e < 8; ++e) big = max(big, abs_bits(x[e]));
    if (kKv == FKV_KV_FP8_E4M3) {
        uint32_t c[4];
        if (quotient2_scale(hs.g) && big <= kQuotient2Max) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 q = quotient2(x[2 * e], x[2 * e + 1], hs.nb, hs.yy);
                // the quotient of a zero loses its sign in the correction step
                c[e] = f32x2_to_e4m3x2(copysignf(q.y, x[2 * e + 1]), copysignf(q.x, x[2 * e]));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * e + 1], hs.g), __fdiv_rn(x[2 * e], hs.g));
        }
        if (row) __stcs(reinterpret_cast<uint2 *>(row) + lane, make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16)));
        return;
    }
    // a scale block is this lane's elements and its neighbour's
    big = max(big, __shfl_xor_sync(half_mask, big, 1));
    const float amax = __uint_as_float(big);
    const bool fast = quotient2_scale(hs.g6) && big <= kQuotient2Max;
    float ratio;
    if (fast) {
        const float q0 = __fmul_rn(amax, hs.y6);
        ratio = __fmaf_rn(__fmaf_rn(q0, -hs.g6, amax), hs.y6, q0);
    } else {
        ratio = __fdiv_rn(amax, hs.g6);
    }
    const uint32_t scale = f32x2_to_e4m3x2(0.f, ratio) & 0xFFu;
    const uint32_t s16 = e4m3x2_to_f16x2(static_cast<uint16_t>(scale));
    const float d = __fmul_rn(__half2float(__ushort_as_half(static_cast<unsigned short>(s16 & 0xFFFFu))), hs.g);
    uint32_t codes = 0;
    if (d > 0.f) {                                             // else: scale 0 or NaN
        uint32_t c[4];
        if (fast && quotient2_scale(d)) {
            const float y = __frcp_rn(d);
            const uint64_t nb = pack2(-d, -d), yy = pack2(y, y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 q = quotient2(x[2 * e], x[2 * e + 1], nb, yy);
                c[e] = f32x2_to_e2m1x2(q.y, q.x);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = f32x2_to_e2m1x2(__fdiv_rn(x[2 * e + 1], d), __fdiv_rn(x[2 * e], d));
        }
        codes = prmt(prmt(c[0], c[1], 0x0040u), prmt(c[2], c[3], 0x0040u), 0x5410u);
    }
    // the row's 8 scale bytes: eight lanes' four blocks make a word
    uint32_t word = scale << (8 * ((lane >> 1) & 3));
    word |= __shfl_xor_sync(half_mask, word, 2);
    word |= __shfl_xor_sync(half_mask, word, 4);
    if (row) {
        __stcs(reinterpret_cast<uint32_t *>(row) + lane, codes);
        if ((lane & 7) == 0) __stcs(reinterpret_cast<uint32_t *>(row + kFp4Codes) + (lane >> 3), word);
    }
}

__device__ __forceinline__ void unpack_bf16x8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = bf16x2_to_f32(w[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
    }
}

template <bool kNeighbours, int kKv>
__global__ void __launch_bounds__(kArBlock, 8)
kv_append_rope_kernel(const AppendRopeParams p) {
    // (several parts only for few tokens: the warps fit 32 bits)
    const uint32_t wid = blockIdx.x * (kArBlock / 32) + threadIdx.x / 32;
    const uint32_t tok = p.parts == 1 ? wid : wid / p.parts;
    const int64_t n = tok;
    grid_dep_wait();                                           // earlier readers of the pool have finished
    grid_dep_launch();
    if (n >= p.n_tokens) return;
    const int first = static_cast<int>(wid - tok * p.parts) * p.rows_per_warp;
    const int last = min(p.heads, first + p.rows_per_warp);
    const int lane = threadIdx.x & 15, hw = (threadIdx.x >> 4) & 1;
    const unsigned half_mask = 0xFFFFu << (16 * hw);
    // rows: the query heads, the key heads, the value heads
    const int k0 = p.hq, v0 = p.hq + p.hkv;
    const int q_end = min(last, k0), k_first = max(first, k0), k_end = min(last, v0), v_first = max(first, v0);
    const uint16_t *qrow = p.q + n * p.qs;
    const uint16_t *krow = p.k + n * p.ks - static_cast<int64_t>(k0) * 128, *vrow = p.v + n * p.vs - static_cast<int64_t>(v0) * 128;
    uint4 u[kArUnroll];
    auto load = [&](int row0, int end, const uint16_t *src) {  // rows row0 + hw, + 2, ... below end
#pragma unroll
        for (int i = 0; i < kArUnroll; ++i) {
            const int row = row0 + 2 * i + hw;
            u[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row < end) u[i] = reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(row) * 128)[lane];
        }
    };
    if (first < q_end) load(first, q_end, qrow);
    else if (k_first < k_end) load(k_first, k_end, krow);
    else load(v_first, last, vrow);

    // the slot's rows in the pools
    int64_t row_base = -1;                                     // of KV head 0, in rows
    if (last > k0) {
        const int64_t slot = __ldg(p.slots + n);
        const uint64_t s = static_cast<uint64_t>(slot);
        if (s < p.total_slots) {
            const uint64_t page = p.page_shift >= 0 ? s >> p.page_shift : s / p.page_size;
            row_base = static_cast<int64_t>(page * p.hkv * p.page_size + (s - page * p.page_size));
        } else if (slot >= 0 && (threadIdx.x & 31) == 0) {
            atomicOr(p.err, FKV_DEVERR_APPEND_SLOT);           // (padding, slot < 0, is only skipped)
        }
    }
    constexpr int kRow = kKv == FKV_KV_BF16 ? 256 : kKv == FKV_KV_FP8_E4M3 ? 128 : kFp4Row;
    auto cached = [&](uint8_t *pool, int h) -> uint8_t * {
        return row_base < 0 ? nullptr : pool + static_cast<uint64_t>(row_base + static_cast<int64_t>(h) * p.page_size) * kRow;
    };

    // this lane's place in the rotation: its elements' pairs j0 .. and, for pairs of
    // halves, whether it holds the second elements and which lane holds the others
    const int nh = p.half >> 3;                                // lanes of first elements
    const bool turned = lane < 2 * nh;
    const bool second = !kNeighbours && lane >= nh;
    const int mate = kNeighbours || !turned ? lane : second ? lane - nh : lane + nh;
    const int j0 = kNeighbours ? 4 * lane : 8 * (second ? mate : lane);
    constexpr int kPairs = kNeighbours ? 4 : 8;                // angles that the lane's elements take
    float c[kPairs], s[kPairs];
    if (first < k_end) {                                       // (a part of value heads needs none)
        // each half-warp (and of two mates each) forms its share
        float2 x[2];
        const int share = kNeighbours ? 2 * hw : 4 * (second ? 1 : 0) + 2 * hw;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[i] = make_float2(1.f, 0.f);                      // an axis that is not there: unturned
            const int j = j0 + share + i;
            if (turned) {
                const int axis = p.axis_map ? __ldg(p.axis_map + j) : 0;
                if (axis < p.n_axes) {
                    x[i] = cos_sin_of(__ldg(p.positions + static_cast<int64_t>(axis) * p.n_tokens + n), __ldg(p.inv_freq + j));
                    x[i].x *= p.rot_scale;
                    x[i].y *= p.rot_scale;
                } else {
                    atomicOr(p.err, FKV_DEVERR_ROPE_AXIS);
                }
            }
        }
        float2 four[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float oc = __shfl_xor_sync(0xffffffffu, x[i].x, 16), os = __shfl_xor_sync(0xffffffffu, x[i].y, 16);
            four[i] = hw ? make_float2(oc, os) : x[i];
            four[2 + i] = hw ? x[i] : make_float2(oc, os);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (kNeighbours) {
                c[i] = four[i].x;
                s[i] = four[i].y;
            } else {
                const float oc = __shfl_sync(0xffffffffu, four[i].x, mate, 16), os = __shfl_sync(0xffffffffu, four[i].y, mate, 16);
                c[i % kPairs] = second ? oc : four[i].x;
                s[i % kPairs] = second ? os : four[i].y;
                c[(4 + i) % kPairs] = second ? four[i].x : oc;
                s[(4 + i) % kPairs] = second ? four[i].y : os;
            }
        }
    }

    // one kind of heads: its rows [row0, end), the first batch loaded already
    auto turn = [&](int row0, int end, const uint16_t *src, const uint4 *weight, auto store) {
        // own' = own * oc + other * os; for neighbours element 2i's other is 2i + 1
        float oc[8], os[8];
        float w[8], ow[8];
        if (weight) {
            unpack_bf16x8(__ldg(weight + lane), w);
            unpack_bf16x8(__ldg(weight + mate), ow);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int j = kNeighbours ? e / 2 : e % kPairs;
            const bool snd = kNeighbours ? e & 1 : second;
            const float we = weight ? w[e] : 1.f, wo = weight ? (kNeighbours ? w[e ^ 1] : ow[e]) : 1.f;
            oc[e] = we * c[j];
            os[e] = snd ? wo * s[j] : -(wo * s[j]);
        }
        for (;; ) {
#pragma unroll
            for (int i = 0; i < kArUnroll; ++i) {
                const int row = row0 + 2 * i + hw;
                const uint4 mine = u[i];
                if (row + kArBatch < end)                      // the next batch's row, in flight from here on
                    u[i] = reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(row + kArBatch) * 128)[lane];
                float a[8], b[8];
                unpack_bf16x8(mine, a);
                if (!kNeighbours) {
                    uint4 theirs;
                    theirs.x = __shfl_sync(0xffffffffu, mine.x, mate, 16);
                    theirs.y = __shfl_sync(0xffffffffu, mine.y, mate, 16);
                    theirs.z = __shfl_sync(0xffffffffu, mine.z, mate, 16);
                    theirs.w = __shfl_sync(0xffffffffu, mine.w, mate, 16);
                    unpack_bf16x8(theirs, b);
                }
                float rs = 1.f;
                if (weight) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], ss);
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    rs = rsqrtf(fmaf(ss, 1.f / 128.f, p.eps));
                }
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float other = kNeighbours ? a[e ^ 1] : b[e];
                    // a lane past rotary_dim keeps its elements apart: 0 times an
                    // infinity in the other one would be a NaN
                    x[e] = rs * (turned ? fmaf(a[e], oc[e], other * os[e]) : a[e] * oc[e]);
                }
                store(row, row < end, x);
            }
            row0 += kArBatch;
            if (row0 >= end) return;
        }
    };
    if (first < q_end) {
        uint16_t *dst = p.q_out + n * p.qos;
        turn(first, q_end, qrow, p.q_weight, [&](int row, bool in, const float (&x)[8]) {
            if (in) __stcs(reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(row) * 128) + lane, pack_bf16x8(x));
        });
        if (k_first < k_end) load(k_first, k_end, krow);
    }
    if (k_first < k_end) {
        turn(k_first, k_end, krow, p.k_weight, [&](int row, bool in, const float (&x)[8]) {
            const int h = min(row, v0 - 1) - k0;
            store_cached<kKv>(in ? cached(p.k_cache, h) : nullptr, lane, half_mask, x, head_scale<kKv>(p.k_scale, h));
        });
        if (v_first < last) load(v_first, last, vrow);
    }
    for (int row0 = v_first; row0 < last; row0 += kArBatch) {
#pragma unroll
        for (int i = 0; i < kArUnroll; ++i) {
            const int row = row0 + 2 * i + hw;
            const uint4 mine = u[i];
            if (row + kArBatch < last)
                u[i] = reinterpret_cast<const uint4 *>(vrow + static_cast<int64_t>(row + kArBatch) * 128)[lane];
            const int h = min(row, p.heads - 1) - v0;
            uint8_t *const dst = row < last ? cached(p.v_cache, h) : nullptr;
            if constexpr (kKv == FKV_KV_BF16) {                    // as they are: a conversion would change a NaN's bits
                if (dst) __stcs(reinterpret_cast<uint4 *>(dst) + lane, mine);
            } else {
                float x[8];
                unpack_bf16x8(mine, x);
                store_cached<kKv>(dst, lane, half_mask, x, head_scale<kKv>(p.v_scale, h));
            }
        }
    }
}

}  // namespace fkv

using namespace fkv;

extern "C" fkv_status kv_append_rope(const void *q, int64_t q_token_stride, int32_t num_q_heads, const void *k,
                                     int64_t k_token_stride, const void *v, int64_t v_token_stride, int32_t num_kv_heads,
                                     void *q_out, int64_t q_out_token_stride, int32_t n_tokens, const void *q_weight,
                                     const void *k_weight, float eps, const int32_t *positions, int32_t n_axes,
                                     const float *inv_freq, const uint8_t *axis_map, int32_t rotary_dim,
                                     int32_t interleaved, float rot_scale, const int64_t *slot_mapping, int32_t kv_dtype,
                                     const float *k_scale, const float *v_scale, void *k_cache, void *v_cache,
                                     int32_t num_pages, int32_t page_size, int32_t head_dim, void *stream) {
    if (n_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || n_axes <= 0 || num_pages <= 0 || page_size <= 0)
        return FKV_ERR_INVALID_ARG;
    if (kv_dtype != FKV_KV_FP8_E4M3 && kv_dtype != FKV_KV_BF16 && kv_dtype != FKV_KV_FP4) return FKV_ERR_INVALID_ARG;
    if (head_dim != 128 || n_axes > kRopeMaxAxes) return FKV_ERR_UNSUPPORTED;
    if (rotary_dim <= 0 || rotary_dim > 128 || rotary_dim % 16) return FKV_ERR_UNSUPPORTED;
    if (num_q_heads > 65535 || num_kv_heads > 32767) return FKV_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(rot_scale)) return FKV_ERR_INVALID_ARG;
    const int64_t qw = static_cast<int64_t>(num_q_heads) * 128, kw = static_cast<int64_t>(num_kv_heads) * 128;
    if (q_token_stride < qw || q_out_token_stride < qw || k_token_stride < kw || v_token_stride < kw)
        return FKV_ERR_INVALID_ARG;
    if ((q_token_stride | q_out_token_stride | k_token_stride | v_token_stride) & 7) return FKV_ERR_INVALID_ARG;
    if (n_tokens == 0) return FKV_OK;
    if (!k || !v || !positions || !inv_freq || !slot_mapping || !k_cache || !v_cache) return FKV_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!q || !q_out)) return FKV_ERR_INVALID_ARG;
    if (kv_dtype != FKV_KV_BF16 && (!k_scale || !v_scale)) return FKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(q_weight) ||
        !aligned16(k_weight) || !aligned16(k_cache) || !aligned16(v_cache))
        return FKV_ERR_INVALID_ARG;
    uint32_t *err = device_error_word();
    const int sms = device_sm_count();
    if (!err || sms <= 0) return FKV_ERR_CUDA;
    AppendRopeParams p;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.qs = q_token_stride;
    p.ks = k_token_stride;
    p.vs = v_token_stride;
    p.qos = q_out_token_stride;
    p.q_weight = static_cast<const uint4 *>(q_weight);
    p.k_weight = static_cast<const uint4 *>(k_weight);
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.axis_map = axis_map;
    p.slots = slot_mapping;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.err = err;
    p.total_slots = static_cast<uint64_t>(num_pages) * static_cast<uint32_t>(page_size);
    p.n_tokens = n_tokens;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.heads = num_q_heads + 2 * num_kv_heads;
    p.n_axes = n_axes;
    p.half = rotary_dim / 2;
    p.page_size = static_cast<uint32_t>(page_size);
    p.page_shift = (page_size & (page_size - 1)) == 0 ? __builtin_ctz(p.page_size) : -1;
    p.eps = eps;
    p.rot_scale = rot_scale;
    // A token's heads are shared out until there are 24 warps per SM, in whole
    // batches: a warp with one batch pays its cos and sin for 8 rows.
    const int most = (p.heads + kArBatch - 1) / kArBatch;
    const int64_t want = (24 * static_cast<int64_t>(sms) + n_tokens - 1) / n_tokens;
    const int parts = static_cast<int>(want < most ? want : most);
    p.rows_per_warp = ((p.heads + parts - 1) / parts + kArBatch - 1) / kArBatch * kArBatch;
    p.parts = (p.heads + p.rows_per_warp - 1) / p.rows_per_warp;
    const int64_t blocks = (static_cast<int64_t>(n_tokens) * p.parts + kArBlock / 32 - 1) / (kArBlock / 32);
    if (blocks > 0x7FFFFFFF) return FKV_ERR_UNSUPPORTED;
    auto go = [&](auto kern) {
        return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kArBlock), 0, static_cast<cudaStream_t>(stream), p);
    };
    auto pick = [&](auto halves, auto neighbours) { return interleaved ? go(neighbours) : go(halves); };
    const cudaError_t e =
        kv_dtype == FKV_KV_FP8_E4M3 ? pick(kv_append_rope_kernel<false, FKV_KV_FP8_E4M3>, kv_append_rope_kernel<true, FKV_KV_FP8_E4M3>)
        : kv_dtype == FKV_KV_BF16   ? pick(kv_append_rope_kernel<false, FKV_KV_BF16>, kv_append_rope_kernel<true, FKV_KV_BF16>)
                                    : pick(kv_append_rope_kernel<false, FKV_KV_FP4>, kv_append_rope_kernel<true, FKV_KV_FP4>);
    return e == cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}
