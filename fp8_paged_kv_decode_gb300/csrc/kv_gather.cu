// kv_gather.cu -- cached tokens read back as bf16 rows.
//
// A prompt's next chunk, or a request that reuses a cached prefix, attends over
// cached tokens outside the decode kernel and needs them dense.  For each listed
// slot and KV head: value * scale in fp32, one rounding to bf16 (BF16 rows are
// copied).  e4m3 codes and e2m1 code * block scale are exact in f16, so the
// product with the head's scale is the only fp32 rounding before bf16's.
//
// Grid of (token groups, KV heads of K then of V): a block reads one head of one
// pool, 8 threads to a row, 16 elements each, so a 4-bit thread reads one scale
// block.  Bound by memory: per (token, KV head) 512 bytes out and 144 (FP4),
// 256 (FP8) or 512 (BF16) in.  A 4-bit thread's row takes 9 bytes of loads, far
// too few in flight to cover their latency, so a thread takes kU tokens and has
// all their slots, then all their rows, in flight together.  262144 tokens of 8
// heads: FP4 277 us with one token a thread, 233 with four (5.9 TB/s; three
// 231, six 246, eight 259), FP8 288 and 253 (6.4 TB/s), BF16 327 with four (6.6 TB/s).
#include "fp4_row.cuh"

namespace fkv {

constexpr int kGatherBlock = 256;
constexpr int kGatherTokens = kGatherBlock / 8;      // rows of a block at a time
constexpr int kGatherMany = 4;                       // tokens per thread of a large call

// Two f16 values times the head's scale, rounded to bf16.
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t f16x2, float g) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&f16x2);
    const float2 f = __half22float2(h);
    return pack_bf16x2(__fmul_rn(f.x, g), __fmul_rn(f.y, g));
}

// The raw bytes of one thread's 16 elements, and their bf16 values.
struct GatherRaw {
    uint4 a, b;
    uint32_t s;
};

template <int kKv>
__device__ __forceinline__ GatherRaw gather_load(const uint8_t *cache, uint64_t row, int chunk) {
    GatherRaw r{};
    if (kKv == FKV_KV_BF16) {
        const uint4 *src = reinterpret_cast<const uint4 *>(cache) + row * 16 + chunk * 2;
        r.a = __ldg(src);
        r.b = __ldg(src + 1);
    } else if (kKv == FKV_KV_FP8_E4M3) {
        r.a = __ldg(reinterpret_cast<const uint4 *>(cache + row * 128) + chunk);
    } else {
        const uint8_t *src = cache + row * kFp4Row;
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(src) + chunk);
        r.a.x = c.x;
        r.a.y = c.y;
        r.s = __ldg(src + kFp4Codes + chunk);
    }
    return r;
}

template <int kKv>
__device__ __forceinline__ void gather_store(uint4 *dst, const GatherRaw &r, float g, bool live) {
    uint4 r0 = make_uint4(0u, 0u, 0u, 0u), r1 = r0;
    if (live) {
        if (kKv == FKV_KV_BF16) {
            r0 = r.a;
            r1 = r.b;
        } else {
            uint32_t f[8];                                 // 16 values in f16, in order
            if (kKv == FKV_KV_FP8_E4M3) {
                const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[2 * j] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[j] & 0xFFFFu));
                    f[2 * j + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[j] >> 16));
                }
            } else {
                const uint32_t s = e4m3_to_f16_pair(r.s);
                uint32_t lo[4], hi[4];
                e2m1x8_to_f16(r.a.x, lo);
                e2m1x8_to_f16(r.a.y, hi);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[j] = mul_f16x2(lo[j], s);
                    f[4 + j] = mul_f16x2(hi[j], s);
                }
            }
            r0 = make_uint4(scaled_bf16x2(f[0], g), scaled_bf16x2(f[1], g), scaled_bf16x2(f[2], g),
                            scaled_bf16x2(f[3], g));
            r1 = make_uint4(scaled_bf16x2(f[4], g), scaled_bf16x2(f[5], g), scaled_bf16x2(f[6], g),
                            scaled_bf16x2(f[7], g));
        }
    }
    __stcs(dst, r0);
    __stcs(dst + 1, r1);
}

struct GatherParams {
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int64_t *slots;
    uint4 *k_out, *v_out;
    uint32_t *err;
    uint64_t total_slots;       // pages x page_size
    uint32_t n_tokens, num_kv_heads, page_size;
    int32_t page_shift;         // log2 of the page size, -1 if it is not a power of two
};

template <int kKv, int kU>
__global__ void __launch_bounds__(kGatherBlock)
kv_gather_kernel(const GatherParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t n0 = blockIdx.x * (kGatherTokens * kU) + threadIdx.x / 8;
    const bool is_v = blockIdx.y >= p.num_kv_heads;
    const uint32_t h = is_v ? blockIdx.y - p.num_kv_heads : blockIdx.y;
    const uint32_t chunk = threadIdx.x & 7;
    const uint8_t *cache = is_v ? p.v_cache : p.k_cache;
    int64_t slot[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const uint32_t n = n0 + u * kGatherTokens;
        slot[u] = n < p.n_tokens ? __ldg(p.slots + n) : -1;
    }
    const float g = kKv == FKV_KV_BF16 ? 1.f : __ldg((is_v ? p.v_scale : p.k_scale) + h);
    GatherRaw raw[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        raw[u] = GatherRaw{};
        const uint64_t s = static_cast<uint64_t>(slot[u]);
        if (s < p.total_slots) {
            const uint64_t page = p.page_shift >= 0 ? s >> p.page_shift : s / p.page_size;
            const uint32_t off = static_cast<uint32_t>(s - page * p.page_size);
            raw[u] = gather_load<kKv>(
                cache, (static_cast<uint64_t>(static_cast<uint32_t>(page)) * p.num_kv_heads + h) * p.page_size + off, chunk);
        } else if (slot[u] >= 0 && chunk == 0) {
            atomicOr(p.err, FKV_DEVERR_GATHER_SLOT);
        }
    }
    const uint32_t row_words = p.num_kv_heads * 16;
    uint4 *out = (is_v ? p.v_out : p.k_out) + static_cast<uint64_t>(n0) * row_words + (h * 16 + chunk * 2);
#pragma unroll
    for (int u = 0; u < kU; ++u)
        if (n0 + u * kGatherTokens < p.n_tokens)
            gather_store<kKv>(out + static_cast<uint64_t>(u * kGatherTokens) * row_words, raw[u], g,
                              static_cast<uint64_t>(slot[u]) < p.total_slots);
}

}  // namespace fkv

using namespace fkv;

extern "C" fkv_status kv_gather(const void *k_cache, const void *v_cache, int32_t kv_dtype, const float *k_scale,
                                const float *v_scale, const int64_t *slots, int32_t n_tokens, void *k_out,
                                void *v_out, int32_t num_pages, int32_t num_kv_heads, int32_t page_size,
                                int32_t head_dim, void *stream) {
    if (n_tokens < 0 || num_pages <= 0 || num_kv_heads <= 0 || page_size <= 0) return FKV_ERR_INVALID_ARG;
    if (kv_dtype != FKV_KV_FP8_E4M3 && kv_dtype != FKV_KV_BF16 && kv_dtype != FKV_KV_FP4) return FKV_ERR_INVALID_ARG;
    if (head_dim != 128 || num_kv_heads > 32767) return FKV_ERR_UNSUPPORTED;          // grid y: K and V heads
    if (n_tokens == 0) return FKV_OK;
    if (!k_cache || !v_cache || !slots || !k_out || !v_out) return FKV_ERR_INVALID_ARG;
    if (kv_dtype != FKV_KV_BF16 && (!k_scale || !v_scale)) return FKV_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out))
        return FKV_ERR_INVALID_ARG;
    uint32_t *err = device_error_word();
    if (!err) return FKV_ERR_CUDA;
    const int sms = device_sm_count();
    if (sms <= 0) return FKV_ERR_CUDA;
    GatherParams p;
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.slots = slots;
    p.k_out = static_cast<uint4 *>(k_out);
    p.v_out = static_cast<uint4 *>(v_out);
    p.err = err;
    p.total_slots = static_cast<uint64_t>(num_pages) * static_cast<uint32_t>(page_size);
    p.n_tokens = static_cast<uint32_t>(n_tokens);
    p.num_kv_heads = static_cast<uint32_t>(num_kv_heads);
    p.page_size = static_cast<uint32_t>(page_size);
    p.page_shift = (page_size & (page_size - 1)) == 0 ? __builtin_ctz(p.page_size) : -1;
    // Several tokens per thread once the grid fills the GPU without that.
    const int64_t rows = 2 * static_cast<int64_t>(n_tokens) * num_kv_heads;
    const bool many = rows >= static_cast<int64_t>(sms) * 8 * kGatherTokens * kGatherMany;
    const int per = kGatherTokens * (many ? kGatherMany : 1);
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(n_tokens) + per - 1) / per),
                    2u * static_cast<unsigned>(num_kv_heads));
    auto go = [&](auto kern) {
        return launch_pdl(kern, grid, dim3(kGatherBlock), 0, static_cast<cudaStream_t>(stream), p);
    };
    auto pick = [&](auto few, auto several) { return many ? go(several) : go(few); };
    const cudaError_t e =
        kv_dtype == FKV_KV_FP8_E4M3
            ? pick(kv_gather_kernel<FKV_KV_FP8_E4M3, 1>, kv_gather_kernel<FKV_KV_FP8_E4M3, kGatherMany>)
        : kv_dtype == FKV_KV_BF16 ? pick(kv_gather_kernel<FKV_KV_BF16, 1>, kv_gather_kernel<FKV_KV_BF16, kGatherMany>)
                                  : pick(kv_gather_kernel<FKV_KV_FP4, 1>, kv_gather_kernel<FKV_KV_FP4, kGatherMany>);
    return e == cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}
