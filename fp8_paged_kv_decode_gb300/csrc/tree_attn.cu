// tree_attn.cu -- attention of drafted tokens, and over a window, on the paged cache.
//
// Request r has n drafted tokens, the last n of its seq_lens[r] cached ones.  Each is
// a query row that sees the committed tokens before them (all of them, or those of a
// window and a few first ones) and the drafted tokens its mask names:
//     out[i][hq] = sum_t softmax_t(sm_scale * q[i][hq] . k_t) v_t   over t seen by i
// A decode step over a window is the same with one token a request.
//
// One block of four warps per (row, query head): each warp takes every fourth token,
// a lane four dims, with a running maximum and sum; the warps' sums are joined at the end.
#include <cmath>

#include "fp4_row.cuh"

namespace fkv {

constexpr int kTreeMaxWords = 4;               // 64-bit words of a row's mask
constexpr int kTreeBlock = 128;

struct TreeParams {
    const __nv_bfloat16 *q;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *indptr, *indices, *seq_lens;
    const int32_t *token_indptr;               // nullptr: one token a request
    const uint64_t *mask;                      // nullptr: a row sees itself
    const uint8_t *abort_mask;
    __nv_bfloat16 *out;
    uint32_t *err;
    int64_t nnz;
    int32_t batch, n_tokens, hq, hkv, pages, page_size, words, window, sinks;
    float scale_log2;
};

template <int kKv>
__device__ __forceinline__ float4 load4(const uint8_t *cache, int64_t row, int lane) {
    if (kKv == FKV_KV_BF16) {
        const uint2 u = reinterpret_cast<const uint2 *>(cache + row * 256)[lane];
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xFFFF0000u));
    }
    uint32_t lo, hi;
    float s = 1.f;
    if (kKv == FKV_KV_FP8_E4M3) {
        const uint32_t u = reinterpret_cast<const uint32_t *>(cache + row * 128)[lane];
        lo = e4m3x2_to_f16x2(static_cast<uint16_t>(u & 0xFFFFu));
        hi = e4m3x2_to_f16x2(static_cast<uint16_t>(u >> 16));
    } else {
        const uint8_t *r = cache + row * kFp4Row;
        uint32_t f[4];
        e2m1x8_to_f16(reinterpret_cast<const uint16_t *>(r)[lane], f);
        lo = f[0];
        hi = f[1];
        const uint32_t s16 = e4m3x2_to_f16x2(r[kFp4Codes + lane / 4]);
        s = __half2float(__ushort_as_half(static_cast<unsigned short>(s16 & 0xFFFFu)));
    }
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
}

template <int kKv>
__global__ void __launch_bounds__(kTreeBlock)
tree_attn_kernel(const TreeParams p) {
    grid_dep_wait();
    grid_dep_launch();
    const int row = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the request of this row: the last one whose rows begin at or before it
    int r = row, t0 = row, t1 = row + 1;
    if (p.token_indptr) {
        int lo = 0, hi = p.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (p.token_indptr[mid] <= row) lo = mid;
            else hi = mid;
        }
        r = lo;
        t0 = p.token_indptr[r];
        t1 = p.token_indptr[r + 1];
        if (t0 < 0 || row < t0 || row >= t1 || t1 > p.n_tokens) return;      // no request's row
    }
    const int n = t1 - t0, len = p.seq_lens[r];
    const int32_t b = p.indptr[r], e = p.indptr[r + 1];
    bool ok = (!p.abort_mask || !p.abort_mask[r]) && len >= n && n <= 64 * p.words && b >= 0 && e >= b && e <= p.nnz &&
              static_cast<int64_t>(e - b) * p.page_size >= len;
    const int ctx = len - n;
    uint64_t m[kTreeMaxWords] = {1, 0, 0, 0};
    if (p.mask)
        for (int w = 0; w < kTreeMaxWords; ++w) m[w] = w < p.words ? p.mask[static_cast<int64_t>(row) * p.words + w] : 0;
    int depth = -1;
    for (int w = 0; w < kTreeMaxWords; ++w) depth += __popcll(m[w]);
    if (depth < 0) depth = 0;
    const int64_t lo64 = p.window ? static_cast<int64_t>(ctx) + depth - p.window + 1 : 0;
    const int lo = lo64 < 0 ? 0 : lo64 > ctx ? ctx : static_cast<int>(lo64);
    const int head = p.window ? min(p.sinks, lo) : 0;
    const int h = hq / (p.hq / p.hkv);
    const __nv_bfloat16 *q = p.q + (static_cast<int64_t>(row) * p.hq + hq) * 128 + 4 * lane;
    const float4 qv = make_float4(__bfloat162float(q[0]), __bfloat162float(q[1]), __bfloat162float(q[2]), __bfloat162float(q[3]));
    const float ks = kKv == FKV_KV_BF16 ? 1.f : p.k_scale[h], vs = kKv == FKV_KV_BF16 ? 1.f : p.v_scale[h];
    const float c = p.scale_log2 * ks;
    float top = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    bool bad = false;
    if (ok) {
        const int seen = head + len - lo;
        for (int i = warp; i < seen; i += kTreeBlock / 32) {
            const int t = i < head ? i : lo + i - head, j = t - ctx;
            const int pg = p.indices[b + t / p.page_size];
            if (pg < 0 || pg >= p.pages) {
                bad = true;
                continue;
            }
            if (j >= 0 && !((m[j >> 6] >> (j & 63)) & 1)) continue;
            const int64_t at = (static_cast<int64_t>(pg) * p.hkv + h) * p.page_size + t % p.page_size;
            const float4 k = load4<kKv>(p.k_cache, at, lane), v = load4<kKv>(p.v_cache, at, lane);
            float z = qv.x * k.x + qv.y * k.y + qv.z * k.z + qv.w * k.w;
#pragma unroll
            for (int x = 16; x; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
            z *= c;
            if (z > top) {
                const float f = exp2f(top - z);
                sum *= f;
                o.x *= f, o.y *= f, o.z *= f, o.w *= f;
                top = z;
            }
            const float w = z == -INFINITY ? 0.f : exp2f(z - top);
            sum += w;
            o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
        }
    }
    __shared__ float4 s_o[kTreeBlock];
    __shared__ float s_top[kTreeBlock / 32], s_sum[kTreeBlock / 32];
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    if (bad && lane == 0) s_bad = 1;
    s_o[threadIdx.x] = o;
    if (lane == 0) s_top[warp] = top, s_sum[warp] = sum;
    __syncthreads();
    if (warp) return;
    float all = -INFINITY, den = 0.f;
    for (int w = 0; w < kTreeBlock / 32; ++w) all = fmaxf(all, s_top[w]);
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < kTreeBlock / 32; ++w) {
        const float f = s_sum[w] == 0.f ? 0.f : exp2f(s_top[w] - all);
        const float4 x = s_o[32 * w + lane];
        if (s_sum[w] == 0.f) continue;
        den = fmaf(f, s_sum[w], den);
        num.x = fmaf(f, x.x, num.x), num.y = fmaf(f, x.y, num.y), num.z = fmaf(f, x.z, num.z), num.w = fmaf(f, x.w, num.w);
    }
    if (s_bad && lane == 0) atomicOr(p.err, FKV_DEVERR_ATTN_PAGE);
    const float g = s_bad || den == 0.f ? 0.f : vs / den;
    if (g == 0.f) num = make_float4(0.f, 0.f, 0.f, 0.f);
    uint2 w;
    w.x = pack_bf16x2(num.x * g, num.y * g);
    w.y = pack_bf16x2(num.z * g, num.w * g);
    reinterpret_cast<uint2 *>(p.out + (static_cast<int64_t>(row) * p.hq + hq) * 128)[lane] = w;
}

namespace {

bool known_kv(int kv) { return kv == FKV_KV_FP8_E4M3 || kv == FKV_KV_BF16 || kv == FKV_KV_FP4; }

fkv_status run(TreeParams p, int kv, void *stream) {
    const dim3 grid(static_cast<unsigned>(p.n_tokens), static_cast<unsigned>(p.hq));
    auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(kTreeBlock), 0, static_cast<cudaStream_t>(stream), p); };
    const cudaError_t e = kv == FKV_KV_FP8_E4M3 ? go(tree_attn_kernel<FKV_KV_FP8_E4M3>)
                          : kv == FKV_KV_BF16   ? go(tree_attn_kernel<FKV_KV_BF16>)
                                                : go(tree_attn_kernel<FKV_KV_FP4>);
    return e == cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}

}  // namespace
}  // namespace fkv

using namespace fkv;

extern "C" size_t paged_tree_attn_workspace_size(int32_t n_tokens, int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                                 int32_t head_dim, int32_t kv_dtype) {
    if (n_tokens < 0 || batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads) return 0;
    if (head_dim != 128 || !known_kv(kv_dtype) || num_q_heads / num_kv_heads > 128) return 0;
    return 256;
}

extern "C" fkv_status paged_tree_attn(const void *q, int32_t n_tokens, int32_t num_q_heads, const void *k_cache,
                                      const void *v_cache, int32_t kv_dtype, const float *k_scale, const float *v_scale,
                                      int32_t num_pages, int32_t num_kv_heads, int32_t page_size, int32_t head_dim,
                                      const int32_t *page_indptr, const int32_t *page_indices, int64_t nnz,
                                      const int32_t *seq_lens, int32_t batch, const int32_t *token_indptr,
                                      const uint64_t *tree_mask, int32_t mask_words, int32_t window, int32_t sinks,
                                      const uint8_t *abort_mask, float sm_scale, void *out, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    const bool tree = token_indptr || tree_mask || mask_words;
    if (n_tokens < 0 || batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_pages <= 0 || nnz < 0) return FKV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads || window < 0 || sinks < 0) return FKV_ERR_INVALID_ARG;
    if (!known_kv(kv_dtype)) return FKV_ERR_INVALID_ARG;
    if (head_dim != 128 || num_q_heads / num_kv_heads > 128 || mask_words > kTreeMaxWords) return FKV_ERR_UNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return FKV_ERR_UNSUPPORTED;
    if (!(sm_scale > 0.f) || !std::isfinite(sm_scale) || mask_words < (tree ? 1 : 0)) return FKV_ERR_INVALID_ARG;
    if (batch == 0 || n_tokens == 0) return FKV_OK;
    if (!q || !k_cache || !v_cache || !page_indptr || !seq_lens || !out || !workspace) return FKV_ERR_INVALID_ARG;
    if (tree ? !token_indptr || !tree_mask : n_tokens != batch) return FKV_ERR_INVALID_ARG;
    if (nnz > 0 && !page_indices) return FKV_ERR_INVALID_ARG;
    if (kv_dtype != FKV_KV_BF16 && (!k_scale || !v_scale)) return FKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return FKV_ERR_INVALID_ARG;
    uint32_t *err = device_error_word();
    if (!err) return FKV_ERR_CUDA;
    if (workspace_bytes < paged_tree_attn_workspace_size(n_tokens, batch, num_q_heads, num_kv_heads, head_dim, kv_dtype))
        return FKV_ERR_INVALID_ARG;
    TreeParams p;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.indptr = page_indptr;
    p.indices = page_indices;
    p.seq_lens = seq_lens;
    p.token_indptr = token_indptr;
    p.mask = tree_mask;
    p.abort_mask = abort_mask;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.err = err;
    p.nnz = nnz;
    p.batch = batch;
    p.n_tokens = n_tokens;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.pages = num_pages;
    p.page_size = page_size;
    p.words = tree ? mask_words : 1;
    p.window = window;
    p.sinks = sinks;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    return run(p, kv_dtype, stream);
}

extern "C" fkv_status paged_window_attn(const void *q, int32_t batch, int32_t num_q_heads, const void *k_cache,
                                        const void *v_cache, int32_t kv_dtype, const float *k_scale, const float *v_scale,
                                        int32_t num_pages, int32_t num_kv_heads, int32_t page_size, int32_t head_dim,
                                        const int32_t *page_indptr, const int32_t *page_indices, int64_t nnz,
                                        const int32_t *seq_lens, int32_t window, int32_t sinks, const uint8_t *abort_mask,
                                        float sm_scale, void *out, void *workspace, size_t workspace_bytes, void *stream) {
    if (window <= 0) return FKV_ERR_INVALID_ARG;
    return paged_tree_attn(q, batch, num_q_heads, k_cache, v_cache, kv_dtype, k_scale, v_scale, num_pages, num_kv_heads,
                           page_size, head_dim, page_indptr, page_indices, nnz, seq_lens, batch, nullptr, nullptr, 0, window,
                           sinks, abort_mask, sm_scale, out, workspace, workspace_bytes, stream);
}
