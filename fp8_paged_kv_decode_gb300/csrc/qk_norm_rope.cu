// qk_norm_rope.cu -- RMS norm of each query and key head and the rotation by
// the token's position, in one pass.
//
//   y = x rsqrt(mean(x^2) + eps) w;  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
// with t = position * inv_freq per pair.  Each row is read and written once:
// bound by memory at 512 bytes a head for prompts, by latency for decode steps.
//
// A warp serves one token, or part of its heads when there are few tokens.  16
// lanes take a head row, 8 elements each, so that both elements of a pair are
// in one lane: lane l holds elements 8l .. 8l + 7 where pairs are neighbours,
// else the four elements 4l .. and their partners rotary_dim / 2 further.  The
// weights are the same for every head, so they go into the rotation's
// coefficients once per token:
//   a' = rs (a wa cos - b wb sin),   b' = rs (b wb cos + a wa sin)
// and a row costs its sum of squares, 12 products and the conversions.  Each
// half-warp has four rows' loads in flight and asks for the next batch's row as
// soon as it has unpacked one.  16411 tokens of 36 heads (302 MB): 118 us with a
// block per token that formed cos and sin before its loads, 54 with a warp per
// token, 51 with the rows asked for ahead, eight resident blocks and streaming
// stores (5.9 TB/s); 64 tokens of 72 heads: 3.4, 2.7 and 2.7 us.
#include <cmath>

#include "fkv_common.cuh"

namespace fkv {

constexpr int kRopeBlock = 128;
constexpr int kRopeUnroll = 4;                 // rows a half-warp has in flight
constexpr int kRopeBatch = 2 * kRopeUnroll;    // rows of a warp's batch
constexpr int kRopeMaxAxes = 8;

struct RopeParams {
    const uint16_t *q, *k;          // bf16
    uint16_t *q_out, *k_out;
    int64_t qs, ks, qos, kos;       // token strides in elements
    const uint4 *q_weight, *k_weight;
    const int32_t *positions;
    const float *inv_freq;
    const uint8_t *axis_map;
    uint32_t *err;
    int32_t n_tokens, hq, heads, parts, rows_per_warp, n_axes, half;
    float eps, rot_scale;
};

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

// A lane's 8 elements (or weights) as the first and second elements of its four
// pairs.  d0, d1: its two groups of four elements, in units of four.
template <bool kNeighbours>
__device__ __forceinline__ void pairs_of(const uint2 u, const uint2 v, float (&a)[4], float (&b)[4]) {
    const float2 u0 = bf16x2_to_f32(u.x), u1 = bf16x2_to_f32(u.y), v0 = bf16x2_to_f32(v.x), v1 = bf16x2_to_f32(v.y);
    if (kNeighbours) {
        a[0] = u0.x, b[0] = u0.y, a[1] = u1.x, b[1] = u1.y;
        a[2] = v0.x, b[2] = v0.y, a[3] = v1.x, b[3] = v1.y;
    } else {
        a[0] = u0.x, a[1] = u0.y, a[2] = u1.x, a[3] = u1.y;
        b[0] = v0.x, b[1] = v0.y, b[2] = v1.x, b[3] = v1.y;
    }
}

template <bool kNeighbours>
__global__ void __launch_bounds__(kRopeBlock, 8)
qk_norm_rope_kernel(const RopeParams p) {
    // (several parts only for few tokens: the warps fit 32 bits)
    const uint32_t wid = blockIdx.x * (kRopeBlock / 32) + threadIdx.x / 32;
    const uint32_t tok = p.parts == 1 ? wid : wid / p.parts;
    const int64_t n = tok;
    grid_dep_wait();
    grid_dep_launch();
    if (n >= p.n_tokens) return;
    const int first = static_cast<int>(wid - tok * p.parts) * p.rows_per_warp;
    const int last = min(p.heads, first + p.rows_per_warp);
    const int lane = threadIdx.x & 15, hw = (threadIdx.x >> 4) & 1;
    // this lane's two groups of four elements; past rotary_dim they are not pairs
    const int np = p.half >> 2;                                // lanes holding pairs
    const bool turned = lane < np;
    const int g0 = kNeighbours ? 2 * lane : turned ? lane : 2 * np + 2 * (lane - np);
    const int g1 = kNeighbours || !turned ? g0 + 1 : lane + np;

    const uint16_t *qrow = p.q + n * p.qs, *krow = p.k + n * p.ks;
    uint2 u[kRopeUnroll], v[kRopeUnroll];
    auto load = [&](int row0, int end, const uint16_t *src) {  // rows row0 + hw, + 2, ... below end
#pragma unroll
        for (int i = 0; i < kRopeUnroll; ++i) {
            const int row = row0 + 2 * i + hw;
            if (row < end) {
                const uint2 *s = reinterpret_cast<const uint2 *>(src + static_cast<int64_t>(row) * 128);
                u[i] = s[g0];
                v[i] = s[g1];
            }
        }
    };
    const int q_end = min(last, p.hq), k_first = max(first, p.hq) - p.hq, k_end = last - p.hq;
    if (first < q_end) load(first, q_end, qrow);
    else load(k_first, k_end, krow);

    // cos and sin of the lane's four pairs, two by each half-warp
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = 4 * lane + 2 * hw + i;
        float2 x = make_float2(1.f, 0.f);                      // an axis that is not there: unturned
        if (turned) {
            const int axis = p.axis_map ? __ldg(p.axis_map + j) : 0;
            if (axis < p.n_axes) {
                x = cos_sin_of(__ldg(p.positions + static_cast<int64_t>(axis) * p.n_tokens + n),
                               __ldg(p.inv_freq + j));
                x.x *= p.rot_scale;
                x.y *= p.rot_scale;
            } else {
                atomicOr(p.err, FKV_DEVERR_ROPE_AXIS);
            }
        }
        const float oc = __shfl_xor_sync(0xffffffffu, x.x, 16), os = __shfl_xor_sync(0xffffffffu, x.y, 16);
        c[i] = hw ? oc : x.x;
        s[i] = hw ? os : x.y;
        c[2 + i] = hw ? x.x : oc;
        s[2 + i] = hw ? x.y : os;
    }

    // one kind of heads: its rows [row0, end), the first batch loaded already
    auto run = [&](int row0, int end, const uint16_t *src, uint16_t *dst, const uint2 *weight) {
        float ac[4], as[4], bc[4], bs[4];
        if (weight) {
            float wa[4], wb[4];
            pairs_of<kNeighbours>(__ldg(weight + g0), __ldg(weight + g1), wa, wb);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ac[i] = wa[i] * c[i];
                as[i] = wa[i] * s[i];
                bc[i] = wb[i] * c[i];
                bs[i] = wb[i] * s[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ac[i] = bc[i] = c[i];
                as[i] = bs[i] = s[i];
            }
        }
        for (;; ) {
#pragma unroll
            for (int i = 0; i < kRopeUnroll; ++i) {
                const int row = row0 + 2 * i + hw;
                float a[4], b[4];
                pairs_of<kNeighbours>(u[i], v[i], a, b);
                if (row + kRopeBatch < end) {                  // the next batch's row, in flight from here on
                    const uint2 *s = reinterpret_cast<const uint2 *>(src + static_cast<int64_t>(row + kRopeBatch) * 128);
                    u[i] = s[g0];
                    v[i] = s[g1];
                }
                float rs = 1.f;
                if (weight) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    rs = rsqrtf(fmaf(ss, 1.f / 128.f, p.eps));
                }
                float x[4], y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // a lane past rotary_dim keeps its elements apart: 0 times an
                    // infinity in the other one would be a NaN
                    x[e] = rs * (turned ? fmaf(a[e], ac[e], -b[e] * bs[e]) : a[e] * ac[e]);
                    y[e] = rs * (turned ? fmaf(b[e], bc[e], a[e] * as[e]) : b[e] * bc[e]);
                }
                if (row < end) {
                    uint2 *d = reinterpret_cast<uint2 *>(dst + static_cast<int64_t>(row) * 128);
                    if (kNeighbours) {
                        __stcs(d + g0, make_uint2(pack_bf16x2(x[0], y[0]), pack_bf16x2(x[1], y[1])));
                        __stcs(d + g1, make_uint2(pack_bf16x2(x[2], y[2]), pack_bf16x2(x[3], y[3])));
                    } else {
                        __stcs(d + g0, make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])));
                        __stcs(d + g1, make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])));
                    }
                }
            }
            row0 += kRopeBatch;
            if (row0 >= end) return;
        }
    };
    if (first < q_end) {
        run(first, q_end, qrow, p.q_out + n * p.qos, reinterpret_cast<const uint2 *>(p.q_weight));
        if (k_first < k_end) load(k_first, k_end, krow);
    }
    if (k_first < k_end) run(k_first, k_end, krow, p.k_out + n * p.kos, reinterpret_cast<const uint2 *>(p.k_weight));
}

}  // namespace fkv

using namespace fkv;

extern "C" fkv_status qk_norm_rope(const void *q, int64_t q_token_stride, int32_t num_q_heads, const void *k,
                                   int64_t k_token_stride, int32_t num_kv_heads, void *q_out,
                                   int64_t q_out_token_stride, void *k_out, int64_t k_out_token_stride,
                                   int32_t n_tokens, const void *q_weight, const void *k_weight, float eps,
                                   const int32_t *positions, int32_t n_axes, const float *inv_freq,
                                   const uint8_t *axis_map, int32_t rotary_dim, int32_t interleaved,
                                   float rot_scale, int32_t head_dim, void *stream) {
    if (n_tokens < 0 || num_q_heads <= 0 || num_kv_heads < 0 || n_axes <= 0) return FKV_ERR_INVALID_ARG;
    if (head_dim != 128 || n_axes > kRopeMaxAxes) return FKV_ERR_UNSUPPORTED;
    if (rotary_dim <= 0 || rotary_dim > 128 || rotary_dim % 16) return FKV_ERR_UNSUPPORTED;
    if (num_q_heads > 65535 || num_kv_heads > 65535) return FKV_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(rot_scale)) return FKV_ERR_INVALID_ARG;
    const int64_t qw = static_cast<int64_t>(num_q_heads) * 128, kw = static_cast<int64_t>(num_kv_heads) * 128;
    if (q_token_stride < qw || q_out_token_stride < qw || k_token_stride < kw || k_out_token_stride < kw)
        return FKV_ERR_INVALID_ARG;
    if ((q_token_stride | q_out_token_stride | k_token_stride | k_out_token_stride) & 7) return FKV_ERR_INVALID_ARG;
    if (n_tokens == 0) return FKV_OK;
    if (!q || !q_out || !positions || !inv_freq) return FKV_ERR_INVALID_ARG;
    if (num_kv_heads > 0 && (!k || !k_out)) return FKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(q_weight) ||
        !aligned16(k_weight))
        return FKV_ERR_INVALID_ARG;
    uint32_t *err = device_error_word();
    const int sms = device_sm_count();
    if (!err || sms <= 0) return FKV_ERR_CUDA;
    RopeParams p;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.qs = q_token_stride;
    p.ks = k_token_stride;
    p.qos = q_out_token_stride;
    p.kos = k_out_token_stride;
    p.q_weight = static_cast<const uint4 *>(q_weight);
    p.k_weight = static_cast<const uint4 *>(k_weight);
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.axis_map = axis_map;
    p.err = err;
    p.n_tokens = n_tokens;
    p.hq = num_q_heads;
    p.heads = num_q_heads + num_kv_heads;
    p.n_axes = n_axes;
    p.half = rotary_dim / 2;
    p.eps = eps;
    p.rot_scale = rot_scale;
    // A token's heads are shared out until there are 24 warps per SM, in whole
    // batches: a warp with one batch pays its cos and sin for 8 rows.
    const int most = (p.heads + kRopeBatch - 1) / kRopeBatch;
    const int64_t want = (24 * static_cast<int64_t>(sms) + n_tokens - 1) / n_tokens;
    const int parts = static_cast<int>(want < most ? want : most);
    p.rows_per_warp = ((p.heads + parts - 1) / parts + kRopeBatch - 1) / kRopeBatch * kRopeBatch;
    p.parts = (p.heads + p.rows_per_warp - 1) / p.rows_per_warp;
    const int64_t blocks = (static_cast<int64_t>(n_tokens) * p.parts + kRopeBlock / 32 - 1) / (kRopeBlock / 32);
    if (blocks > 0x7FFFFFFF) return FKV_ERR_UNSUPPORTED;
    auto go = [&](auto kern) {
        return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kRopeBlock), 0,
                          static_cast<cudaStream_t>(stream), p);
    };
    const cudaError_t e = interleaved ? go(qk_norm_rope_kernel<true>) : go(qk_norm_rope_kernel<false>);
    return e == cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}
