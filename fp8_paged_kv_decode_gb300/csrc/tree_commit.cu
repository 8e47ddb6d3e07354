// tree_commit.cu -- the accepted drafted tokens' rows moved to where they belong.
//
// Request r has n drafted tokens, the last n of its seq_lens[r] cached ones; of them
// the verification kept a path, accepted[r][0 .. count): strictly increasing, so the
// i-th kept one lies at or behind position ctx + i, where the next step expects it.
// Rows move in that order: a move's target was read by an earlier move or is not read
// at all, and within a round of moves every row is loaded before one is stored.
//
// A warp serves one (request, KV head) of K or V.  Its lanes look up 32 kept tokens'
// rows at a time; then 8 (FP8), 16 (BF16) or 9 (FP4) lanes copy a row, several rows in
// one access.  Bound by latency: a few rows of 72 to 256 bytes per warp behind four
// dependent loads (lengths, list, page, row).  One block more gives the pages past the
// kept lengths back, in the order that makes the free list what it was before.
#include "fkv_common.cuh"

namespace fkv {

constexpr int kCommitBlock = 256;

struct CommitParams {
    uint8_t *k_cache, *v_cache;
    const int32_t *indptr, *indices, *seq_lens, *token_indptr, *accepted, *counts;
    const uint8_t *abort_mask;
    int32_t *lens_out, *free_pages, *free_left;
    const int32_t *free_count;
    uint32_t *page_tags, *err;
    int64_t nnz, units;                        // units: (request, KV head, K or V)
    int32_t batch, n_tokens, max_accepted, pages, hkv, page_size, num_free;
};

// A request's rows, as far as its arrays make sense.
struct CommitRequest {
    int32_t ctx, len, row, count;              // committed and all tokens, first page-table entry, kept drafts
    bool live;                                 // false: left as it is
};

__device__ __forceinline__ CommitRequest commit_request(const CommitParams &p, int r) {
    CommitRequest c{};
    const int32_t t0 = __ldg(p.token_indptr + r), t1 = __ldg(p.token_indptr + r + 1);
    const int32_t b = __ldg(p.indptr + r), e = __ldg(p.indptr + r + 1);
    c.len = __ldg(p.seq_lens + r);
    c.count = __ldg(p.counts + r);
    const bool alive = !p.abort_mask || __ldg(p.abort_mask + r) == 0;
    c.row = b;
    c.live = alive && t0 >= 0 && t1 >= t0 && t1 <= p.n_tokens && c.len >= t1 - t0 && b >= 0 && e >= b && e <= p.nnz &&
             static_cast<int64_t>(e - b) * p.page_size >= c.len;
    c.ctx = c.len - (t1 - t0);
    return c;
}

// Whether part `lane` of `lanes` of a live request's kept list and drafted tokens' pages
// are what they have to be.
__device__ __forceinline__ bool commit_valid(const CommitParams &p, const CommitRequest &c, int r, int lane, int lanes) {
    const int n = c.len - c.ctx;
    bool ok = c.count >= 0 && c.count <= n && c.count <= p.max_accepted;
    if (!ok || n == 0) return ok;
    const int32_t *list = p.accepted + static_cast<int64_t>(r) * p.max_accepted;
    for (int i = lane; i < c.count; i += lanes) {
        const int a = __ldg(list + i), before = i ? __ldg(list + i - 1) : -1;
        ok &= a > before && a < n;
    }
    const int last = (c.len - 1) / p.page_size;
    for (int j = c.ctx / p.page_size + lane; j <= last; j += lanes)
        ok &= static_cast<uint32_t>(__ldg(p.indices + c.row + j)) < static_cast<uint32_t>(p.pages);
    return ok;
}

template <typename V, int kLanes>                              // kLanes x V: a row
__device__ __forceinline__ void commit_move(uint8_t *pool, const CommitParams &p, const CommitRequest &c, int r, int h, int lane) {
    constexpr int kRows = 32 / kLanes;                         // rows of an access
    constexpr int kUnroll = 4;
    const int32_t *list = p.accepted + static_cast<int64_t>(r) * p.max_accepted;
    const int sub = lane / kLanes, col = lane - sub * kLanes;
    auto place = [&](int t) {                                  // the row of token t
        const int64_t pg = __ldg(p.indices + c.row + t / p.page_size);
        return (pg * p.hkv + h) * p.page_size + t % p.page_size;
    };
    for (int base = 0; base < c.count; base += 32) {
        const int i = base + lane;
        int64_t src = 0, dst = 0;                              // equal: nothing to move
        if (i < c.count) {
            const int a = __ldg(list + i);
            if (a != i) {
                src = place(c.ctx + a);
                dst = place(c.ctx + i);
            }
        }
        const int rows = min(32, c.count - base);
        for (int k = 0; k < rows; k += kRows * kUnroll) {
            V v[kUnroll];
            int64_t to[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int j = k + u * kRows + sub;
                const int64_t s = __shfl_sync(0xffffffffu, src, j & 31), d = __shfl_sync(0xffffffffu, dst, j & 31);
                to[u] = sub < kRows && j < rows && s != d ? d * kLanes + col : -1;
                if (to[u] >= 0) v[u] = reinterpret_cast<const V *>(pool)[s * kLanes + col];
            }
            __syncwarp();                                      // every row of the round is loaded
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (to[u] >= 0) reinterpret_cast<V *>(pool)[to[u]] = v[u];
            __syncwarp();
        }
    }
}

// The pages past the kept lengths, given back so that the next step takes them from the
// top of the list in the order in which this one did.
__device__ __forceinline__ void commit_release(const CommitParams &p) {
    __shared__ int s_warp[kCommitBlock / 32];
    __shared__ int s_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int have = min(max(*p.free_count, 0), p.num_free);
    int64_t total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int64_t before = 0;                                    // pages of the chunks so far
        for (int base = 0; base < p.batch; base += kCommitBlock) {
            const int r = base + tid;
            int back = 0, first = 0, row = 0;
            if (r < p.batch) {
                const CommitRequest c = commit_request(p, r);
                if (c.live && commit_valid(p, c, r, 0, 1)) {
                    const int64_t s = p.page_size;
                    first = static_cast<int>((c.ctx + c.count + s - 1) / s);
                    back = static_cast<int>((c.len + s - 1) / s) - first;
                    row = c.row;
                }
            }
            int x = back;                                      // inclusive scan over the block
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) s_warp[warp] = x;
            __syncthreads();
            if (tid == 0) {
                int run = 0;
                for (int w = 0; w < kCommitBlock / 32; ++w) {
                    const int y = s_warp[w];
                    s_warp[w] = run;
                    run += y;
                }
                s_base = run;
            }
            __syncthreads();
            if (pass && total <= p.num_free - have) {
                const int64_t at = have + total - 1 - (before + s_warp[warp] + x - back);
                for (int k = 0; k < back; ++k) {
                    const int32_t pg = __ldg(p.indices + row + first + k);
                    p.free_pages[at - k] = pg;
                    if (p.page_tags) p.page_tags[pg] += 1;
                }
            }
            before += s_base;
            __syncthreads();                                   // s_warp and s_base are read
        }
        total = before;
    }
    if (tid == 0) {
        const bool fits = total <= p.num_free - have;
        *p.free_left = have + (fits ? static_cast<int>(total) : 0);
        if (!fits) atomicOr(p.err, FKV_DEVERR_TREE);
    }
}

template <int kKv>
__global__ void __launch_bounds__(kCommitBlock)
kv_tree_commit_kernel(const CommitParams p, bool release) {
    grid_dep_wait();                                           // the verification's results, earlier readers of the pool
    grid_dep_launch();
    if (release && blockIdx.x == 0) {
        commit_release(p);
        return;
    }
    const int64_t unit = static_cast<int64_t>(blockIdx.x - (release ? 1 : 0)) * (kCommitBlock / 32) + threadIdx.x / 32;
    if (unit >= p.units) return;
    const int lane = threadIdx.x & 31;
    const int r = static_cast<int>(unit / (2 * p.hkv)), hv = static_cast<int>(unit - static_cast<int64_t>(r) * 2 * p.hkv);
    const bool is_v = hv >= p.hkv;
    const int h = is_v ? hv - p.hkv : hv;
    const CommitRequest c = commit_request(p, r);
    if (!c.live) return;
    if (!__all_sync(0xffffffffu, commit_valid(p, c, r, lane, 32))) {
        if (hv == 0 && lane == 0) atomicOr(p.err, FKV_DEVERR_TREE);
        return;
    }
    if (hv == 0 && lane == 0) p.lens_out[r] = c.ctx + c.count;
    uint8_t *pool = is_v ? p.v_cache : p.k_cache;
    if (kKv == FKV_KV_FP8_E4M3) commit_move<uint4, 8>(pool, p, c, r, h, lane);
    else if (kKv == FKV_KV_BF16) commit_move<uint4, 16>(pool, p, c, r, h, lane);
    else commit_move<uint2, 9>(pool, p, c, r, h, lane);
}

}  // namespace fkv

using namespace fkv;

extern "C" fkv_status kv_tree_commit(void *k_cache, void *v_cache, int32_t kv_dtype, int32_t num_pages, int32_t num_kv_heads,
                                     int32_t page_size, int32_t head_dim, const int32_t *page_indptr,
                                     const int32_t *page_indices, int64_t nnz, const int32_t *seq_lens, int32_t batch,
                                     const int32_t *token_indptr, int32_t n_tokens, const int32_t *accepted,
                                     int32_t max_accepted, const int32_t *accepted_counts, const uint8_t *abort_mask,
                                     int32_t *lens_out, int32_t *free_pages, int32_t num_free, const int32_t *free_count,
                                     int32_t *free_left, uint32_t *page_tags, void *stream) {
    if (batch < 0 || n_tokens < 0 || num_pages <= 0 || num_kv_heads <= 0 || page_size <= 0 || nnz < 0 || max_accepted < 0 ||
        num_free < 0)
        return FKV_ERR_INVALID_ARG;
    if (kv_dtype != FKV_KV_FP8_E4M3 && kv_dtype != FKV_KV_BF16 && kv_dtype != FKV_KV_FP4) return FKV_ERR_INVALID_ARG;
    if (head_dim != 128 || num_kv_heads > 32767) return FKV_ERR_UNSUPPORTED;
    const bool release = free_pages || free_count || free_left || page_tags || num_free;
    if (release && (!free_count || !free_left || (num_free > 0 && !free_pages))) return FKV_ERR_INVALID_ARG;
    if (batch == 0 && !release) return FKV_OK;
    if (batch > 0) {
        if (!k_cache || !v_cache || !page_indptr || !seq_lens || !token_indptr || !accepted_counts || !lens_out)
            return FKV_ERR_INVALID_ARG;
        if ((nnz > 0 && !page_indices) || (max_accepted > 0 && !accepted)) return FKV_ERR_INVALID_ARG;
        // read by a request's other warps while one of them writes its kept length
        if (lens_out == seq_lens || lens_out == accepted_counts || lens_out == accepted) return FKV_ERR_INVALID_ARG;
        if (!aligned16(k_cache) || !aligned16(v_cache)) return FKV_ERR_INVALID_ARG;
    }
    uint32_t *err = device_error_word();
    if (!err) return FKV_ERR_CUDA;
    CommitParams p;
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.indptr = page_indptr;
    p.indices = page_indices;
    p.seq_lens = seq_lens;
    p.token_indptr = token_indptr;
    p.accepted = accepted;
    p.counts = accepted_counts;
    p.abort_mask = abort_mask;
    p.lens_out = lens_out;
    p.free_pages = free_pages;
    p.free_left = free_left;
    p.free_count = free_count;
    p.page_tags = page_tags;
    p.err = err;
    p.nnz = nnz;
    p.units = static_cast<int64_t>(batch) * num_kv_heads * 2;
    p.batch = batch;
    p.n_tokens = n_tokens;
    p.max_accepted = max_accepted;
    p.pages = num_pages;
    p.hkv = num_kv_heads;
    p.page_size = page_size;
    p.num_free = num_free;
    const int64_t blocks = (p.units + kCommitBlock / 32 - 1) / (kCommitBlock / 32) + (release ? 1 : 0);
    if (blocks > 0x7FFFFFFF) return FKV_ERR_UNSUPPORTED;
    auto go = [&](auto kern) {
        return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kCommitBlock), 0, static_cast<cudaStream_t>(stream), p,
                          release);
    };
    const cudaError_t e = kv_dtype == FKV_KV_FP8_E4M3 ? go(kv_tree_commit_kernel<FKV_KV_FP8_E4M3>)
                          : kv_dtype == FKV_KV_BF16   ? go(kv_tree_commit_kernel<FKV_KV_BF16>)
                                                      : go(kv_tree_commit_kernel<FKV_KV_FP4>);
    return e == cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}
