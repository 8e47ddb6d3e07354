// qk_norm_rope.cu -- RMS norm of each query and key head and the rotation by
// the token's position, in one pass.
//
//   y = x rsqrt(mean(x^2) + eps) w;  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
// with t = position * inv_freq per pair.  Each row is read and written once:
// bound by memory at 512 bytes a head for prompts, by latency for decode steps.
//
// A block serves one token (or part of its heads): its threads first form the
// token's cos and sin once, for all heads, in shared memory; then 16 threads
// take a head row, 8 elements (16 bytes) each.
#include <cmath>

#include "fkv_common.cuh"

namespace fkv {

constexpr int kRopeBlock = 256;
constexpr int kRopeRows = kRopeBlock / 16;     // head rows a block has in flight
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
    int32_t n_tokens, hq, heads, rows_per_block, n_axes, half, interleaved;
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

__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

__global__ void __launch_bounds__(kRopeBlock)
qk_norm_rope_kernel(const RopeParams p) {
    __shared__ float2 cs[64];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t n = blockIdx.x;
    const int lane = threadIdx.x & 15;
    const int first = blockIdx.y * p.rows_per_block;
    const int last = min(p.heads, first + p.rows_per_block);
    if (threadIdx.x < p.half) {
        const int j = threadIdx.x;
        const int axis = p.axis_map ? __ldg(p.axis_map + j) : 0;
        float2 v = make_float2(1.f, 0.f);                      // an axis that is not there: unturned
        if (axis < p.n_axes) {
            v = cos_sin_of(__ldg(p.positions + static_cast<int64_t>(axis) * p.n_tokens + n), __ldg(p.inv_freq + j));
            v.x *= p.rot_scale;
            v.y *= p.rot_scale;
        } else {
            atomicOr(p.err, FKV_DEVERR_ROPE_AXIS);
        }
        cs[j] = v;
    }
    __syncthreads();
    // this thread's 8 elements 8 lane .. 8 lane + 7 and where they turn
    const bool turned = 8 * lane < 2 * p.half;
    const int step = p.half >> 3;                              // lanes between the two parts of a pair
    const bool upper = !p.interleaved && turned && lane >= step;
    const int partner = p.interleaved || !turned ? lane : upper ? lane - step : lane + step;
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
        if (turned) {
            const int j = p.interleaved ? 4 * lane + (i >> 1) : 8 * (upper ? lane - step : lane) + i;
            const float2 v = cs[j];
            c[i] = v.x;
            // out = y c + partner's y s: the first of a pair takes -sin
            s[i] = (p.interleaved ? (i & 1) != 0 : upper) ? v.y : -v.y;
        }
    }
    for (int row = first + threadIdx.x / 16; row < last; row += kRopeRows) {
        const bool is_k = row >= p.hq;
        const int h = is_k ? row - p.hq : row;
        const uint16_t *src = (is_k ? p.k + n * p.ks : p.q + n * p.qs) + h * 128;
        uint16_t *dst = (is_k ? p.k_out + n * p.kos : p.q_out + n * p.qos) + h * 128;
        const uint4 *w = is_k ? p.k_weight : p.q_weight;
        const uint4 v = *(reinterpret_cast<const uint4 *>(src) + lane);
        const unsigned mask = 0xFFFFu << (threadIdx.x & 16);
        float x[8], y[8], z[8];
        unpack8(v, x);
        uint4 u;                                               // the partner's elements
        const int from = (threadIdx.x & 16) + partner;
        u.x = __shfl_sync(mask, v.x, from);
        u.y = __shfl_sync(mask, v.y, from);
        u.z = __shfl_sync(mask, v.z, from);
        u.w = __shfl_sync(mask, v.w, from);
        unpack8(u, z);
        if (w) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(mask, ss, o);
            const float rs = rsqrtf(fmaf(ss, 1.f / 128.f, p.eps));
            float wx[8], wz[8];
            unpack8(__ldg(w + lane), wx);
            unpack8(__ldg(w + partner), wz);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = x[i] * rs * wx[i];
                z[i] = z[i] * rs * wz[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float other = p.interleaved ? x[i ^ 1] : z[i];
            y[i] = turned ? fmaf(x[i], c[i], other * s[i]) : x[i];
        }
        *(reinterpret_cast<uint4 *>(dst) + lane) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                             pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    }
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
    p.interleaved = interleaved != 0;
    p.eps = eps;
    p.rot_scale = rot_scale;
    // few tokens: several blocks share a token's heads
    int parts = 1;
    while (static_cast<int64_t>(n_tokens) * parts < 2 * sms && parts * kRopeRows < p.heads) ++parts;
    p.rows_per_block = ((p.heads + parts - 1) / parts + kRopeRows - 1) / kRopeRows * kRopeRows;
    parts = (p.heads + p.rows_per_block - 1) / p.rows_per_block;
    const cudaError_t e = launch_pdl(qk_norm_rope_kernel, dim3(static_cast<unsigned>(n_tokens),
                                                               static_cast<unsigned>(parts)),
                                     dim3(kRopeBlock), 0, static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}
