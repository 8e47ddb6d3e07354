// tree_attn.cuh -- what the kernels of tree and window attention share: which tiles a
// request has, which rows see a token, equal shares of all tiles, and the joining of units
// that several shares have parts of.
//
// The n drafted tokens of a request and the G query heads of a KV head read the same K and V:
// a unit is (request, KV head, rows of some of its drafted tokens), a tile kTok of the tokens
// that its rows see.  The tiles of all units, laid end to end, are cut into equal shares.
#pragma once

#include "fp4_row.cuh"

namespace fkv {

constexpr int kTreeMaxWords = 4;               // 64-bit words of a row's mask
constexpr float kTreeNone = -3e38f;            // the reference of a row that has seen nothing
// log2 of a moved reference's largest weight, and of any weight: f16 words take all of f16's range; of BF16 ones, which have
// fp32's, none is above 1, so that no sum over V of any size overflows that the output does not.
template <int kKv>
constexpr float kTreeTop = kKv == FKV_KV_BF16 ? -6.f : 10.f;
template <int kKv>
constexpr float kTreeMost = kKv == FKV_KV_BF16 ? 0.f : 15.9f;
// The reference that a largest logit of z asks for.  Past 2^27 fp32 neighbours are 16 and more apart, and z - 10 may round
// to z - 16, whose weight of 2^16 f16 does not hold: there it is z itself.
template <int kKv>
__device__ __forceinline__ float tree_reference(float z) {
    const float r = __fsub_rn(z, kTreeTop<kKv>);
    return __fsub_rn(z, r) > kTreeMost<kKv> ? z : r;
}
// Whether an exponent c s - ref needs c s rounded first, as the reference's logit was.  One fused operation leaves
// that rounding in the exponent, up to half an fp32 step of the logit: 1/16 below 2^20, 2^9 at 1e10, where weights would
// overflow or vanish.  (The compiler fuses the packed mul.rn and add.rn of PTX too; __fmul_rn and __fadd_rn stay apart.)
__device__ __forceinline__ bool reference_far(float ref) { return fabsf(ref) >= 0x1p20f && ref > kTreeNone; }
constexpr uint32_t kAll = 0xffffffffu;

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
    // [2 shares][rows][128], [2 shares][rows]: sums of units that are cut, their references and weights' sums (sum < 0: a
    // bad page); [shares] the unit whose last part a share has: first share (-1: none), token, tokens, KV head
    float *part_o;
    float2 *part_ml;
    int4 *joins;
    int64_t nnz;
    int32_t batch, n_tokens, hq, hkv, group, pages, page_size, words, window, sinks;
    float scale_log2;
};

// ---------------------------------------------------------------------------
// geometry
// ---------------------------------------------------------------------------
struct TreeRequest {
    int32_t t0, n, len, row;                   // first query token, drafted and all tokens, first page-table entry
    bool live, rows;                           // has work; its rows are rows of q
};

__device__ __forceinline__ TreeRequest tree_request(const TreeParams &p, int r) {
    TreeRequest q{};
    if (r >= p.batch) return q;
    int t0 = r, t1 = r + 1;
    if (p.token_indptr) {
        t0 = __ldg(p.token_indptr + r);
        t1 = __ldg(p.token_indptr + r + 1);
    }
    const int32_t b = __ldg(p.indptr + r), e = __ldg(p.indptr + r + 1);
    q.len = __ldg(p.seq_lens + r);
    const bool alive = !p.abort_mask || __ldg(p.abort_mask + r) == 0;
    q.t0 = t0;
    q.row = b;
    q.rows = t0 >= 0 && t1 >= t0 && t1 <= p.n_tokens;
    q.n = q.rows ? t1 - t0 : 0;
    q.live = q.n > 0 && alive && q.len >= q.n && q.n <= 64 * p.words && b >= 0 && e >= b && e <= p.nnz &&
             static_cast<int64_t>(e - b) * p.page_size >= q.len;
    return q;
}

// The tiles of a live request: those over the first tokens, if there are pages between (which
// are not read: they may be given back, their entries stale), then those from `start` on, the
// page of the first token that a row at depth 0 sees.
struct TreeSpan {
    int32_t start, sink_tiles, head, tiles;
};
template <int kTok>                            // tokens of a tile
__device__ __forceinline__ TreeSpan tree_span(const TreeParams &p, const TreeRequest &q) {
    TreeSpan s{0, 0, 0, 0};
    const int32_t ctx = q.len - q.n;
    if (p.window && ctx >= p.window) {
        const int32_t lo = ctx - p.window + 1;
        s.start = lo - lo % p.page_size;
        s.head = min(p.sinks, lo);
        s.sink_tiles = s.head / kTok + (s.head % kTok != 0);
        if (s.start < static_cast<int64_t>(s.head) + p.page_size) s = TreeSpan{0, 0, 0, 0};    // (start begins a page)
    }
    s.tiles = s.sink_tiles + (q.len - s.start - 1) / kTok + 1;
    return s;
}

// What a share has of a unit.
struct TreeUnit {
    int32_t tb, te;                            // its tiles; te < 0: there is no more work
    int32_t tok0, ntok;                        // the rows' tokens
    int32_t ctx, len;
    int32_t start, sink_tiles, head;
    int32_t whole[3];                          // tiles [0, whole[0]) and [whole[1], whole[2]) are seen by every row
    int32_t row, h;                            // first page-table entry, KV head
    int32_t slot;                              // of its partial sums; -1: the whole unit is here
    int32_t bad;                               // a page outside the pool
    int32_t odd;                               // NaN or infinities in V that not every row sees
};
template <int kTok>
__device__ __forceinline__ uint32_t tile_at(const TreeUnit &u, int i) {
    return i < u.sink_tiles ? static_cast<uint32_t>(i) * kTok : u.start + static_cast<uint32_t>(i - u.sink_tiles) * kTok;
}
__device__ __forceinline__ uint32_t tile_end(const TreeUnit &u, int i) { return i < u.sink_tiles ? u.head : u.len; }
// Sets u.whole, with the unit's spans and lengths in place: tiles of committed tokens that lie
// within every row's window, or among the first tokens.
template <int kTok>
__device__ __forceinline__ void unit_whole(const TreeParams &p, TreeUnit &u) {
    const int32_t far = p.window && u.len > p.window ? u.len - p.window : 0;       // the deepest row's first token, at most
    u.whole[2] = u.ctx > u.start ? u.sink_tiles + (u.ctx - u.start) / kTok : 0;
    u.whole[1] = u.sink_tiles + (far > u.start ? (far - u.start - 1) / kTok + 1 : 0);
    u.whole[0] = p.window ? min(u.sink_tiles ? u.sink_tiles : u.whole[2], min(p.sinks, u.ctx) / kTok) : 0;
}
// Whether every row sees every token of tile i.
__device__ __forceinline__ bool tile_whole(const TreeUnit &u, int i) { return i < u.whole[0] || (i >= u.whole[1] && i < u.whole[2]); }

// ---------------------------------------------------------------------------
// which rows see a token
// ---------------------------------------------------------------------------
// Word w of a row's mask, without the bits of tokens that are not there (`n` are): they name
// nothing, and count for no depth, so no row is deeper than unit_whole takes for the deepest.
__device__ __forceinline__ uint64_t mask_word(const uint64_t *m, int w, int n) {
    const int left = n - 64 * w;
    return __ldg(m + w) & (left >= 64 ? ~0ull : left > 0 ? (1ull << left) - 1 : 0ull);
}
struct RowSight {
    uint64_t word;                             // the row's mask word of the token asked for
    int32_t lo;                                // its first committed token apart from the first ones
};
// Of drafted row `tok` (of the call), for tokens of mask word `w`.
__device__ __forceinline__ RowSight row_sight(const TreeParams &p, const TreeUnit &u, int tok, int w) {
    RowSight s{w == 0 ? 1ull : 0ull, 0};
    int bits = 1;
    if (p.mask) {
        const uint64_t *m = p.mask + static_cast<int64_t>(tok) * p.words;
        s.word = w < p.words ? mask_word(m, w, u.len - u.ctx) : 0ull;
        if (p.window) {
            bits = 0;
            for (int i = 0; i < p.words; ++i) bits += __popcll(mask_word(m, i, u.len - u.ctx));
        }
    }
    if (p.window) s.lo = static_cast<int32_t>(static_cast<int64_t>(u.ctx) + max(bits - 1, 0) - p.window + 1 > 0 ? static_cast<int64_t>(u.ctx) + max(bits - 1, 0) - p.window + 1 : 0);
    return s;
}
// (end: of the tile's tokens; those over the first ones may reach into the others' places)
__device__ __forceinline__ bool sees(const TreeParams &p, const TreeUnit &u, const RowSight &s, uint32_t t, uint32_t end) {
    if (t >= end) return false;
    if (t >= static_cast<uint32_t>(u.ctx)) return (s.word >> ((t - u.ctx) & 63)) & 1;
    return !p.window || t < static_cast<uint32_t>(p.sinks) || t >= static_cast<uint32_t>(s.lo);
}
__device__ __forceinline__ int word_of(const TreeUnit &u, uint32_t t) {
    return t >= static_cast<uint32_t>(u.ctx) ? static_cast<int>((t - u.ctx) >> 6) : 0;
}
// Which of the 32 tokens from t0 on row `tok` (of the call; -1: none) sees, of a tile's up to `end`.
__device__ __forceinline__ uint32_t seen_of(const TreeParams &p, const TreeUnit &u, int tok, uint32_t t0, uint32_t end) {
    if (tok < 0) return 0u;
    auto below = [t0](int64_t x) {                                 // tokens before x
        const int64_t d = x - t0;
        return d >= 32 ? kAll : d <= 0 ? 0u : (1u << d) - 1u;
    };
    const int64_t at = static_cast<int64_t>(t0) - u.ctx;           // of the drafted tokens
    uint64_t lo = 0, hi = 0;                                       // the mask words of tokens at and at + 32
    int bits = 1;
    if (p.mask) {
        const uint64_t *m = p.mask + static_cast<int64_t>(tok) * p.words;
        bits = 0;
#pragma unroll
        for (int i = 0; i < kTreeMaxWords; ++i) {
            const uint64_t w = i < p.words ? mask_word(m, i, u.len - u.ctx) : 0ull;
            bits += __popcll(w);
            if (at >= 64 * i && at < 64 * i + 64) lo = w;
            if (at + 63 >= 64 * i && at + 63 < 64 * i + 64) hi = w;
        }
    } else {
        lo = at >= 0 && at < 64 ? 1ull : 0ull;
        hi = at + 63 >= 0 && at + 63 < 64 ? 1ull : 0ull;
    }
    const int sh = static_cast<int>(at & 63);
    const uint32_t drafted = static_cast<uint32_t>((lo >> sh) | (sh ? hi << (64 - sh) : 0ull));
    uint32_t old = below(u.ctx);
    if (p.window) old &= below(p.sinks) | ~below(static_cast<int64_t>(u.ctx) + max(bits - 1, 0) - p.window + 1);
    return (old | (drafted & ~below(u.ctx))) & below(end);
}

// ---------------------------------------------------------------------------
// values
// ---------------------------------------------------------------------------
// Queries become f16 with a power of two that puts the largest of them into [2^15, 2^16): BF16's 8 bits end at 65280 there,
// below f16's 65504, and 2^-32 of the largest keeps its last bit at 2^-24, f16's lowest.
struct QueryPower {
    float up, down;                            // 2^k and 2^-k
};
// For a largest element with these bits (BF16, no sign).  Zeros, infinities and NaN stay what they are.
__device__ __forceinline__ QueryPower query_power(uint32_t big) {
    int e = static_cast<int>(big >> 7);
    if (e == 0 || e == 255) e = 142;
    e = max(e, 16);
    return {__uint_as_float(static_cast<uint32_t>(269 - e) << 23), __uint_as_float(static_cast<uint32_t>(e - 15) << 23)};
}
// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    lo = e4m3x2_to_f16x2(static_cast<uint16_t>(w & 0xFFFFu));
    hi = e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
}
// A V value that is NaN or infinite, as the cache holds it; else 0.
template <int kKv>
__device__ __forceinline__ float odd_value(const TreeParams &p, const TreeUnit &u, uint32_t t, int dim) {
    const int64_t pg = __ldg(p.indices + u.row + t / p.page_size);
    if (pg < 0 || pg >= p.pages) return 0.f;
    const int64_t row = (pg * p.hkv + u.h) * p.page_size + t % p.page_size;
    float v;
    if (kKv == FKV_KV_BF16) {
        v = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p.v_cache)[row * 128 + dim]) << 16);
    } else {
        const uint32_t b = kKv == FKV_KV_FP8_E4M3 ? p.v_cache[row * 128 + dim] : p.v_cache[row * kFp4Row + kFp4Codes + dim / 16];
        v = (b & 0x7Fu) == 0x7Fu ? __int_as_float(0x7FC00000) : 0.f;
    }
    return isfinite(v) ? 0.f : v;
}

// A V row in its stage, of a tile that not every row sees whole: rows of no token, NaN and
// infinities become zeros, since a weight of zero would not take them out of a product.
// Returns whether there were NaN or infinities.  A pass of its own over these few tiles keeps
// the conversions small: with both forms of them in the loop every tile paid for the tests
// (64 requests, window of 4096: 173 us, 120 without).
template <int kKv>
__device__ __forceinline__ bool clean_v(uint32_t stage, int tok, bool valid) {
    bool odd = false;
    constexpr int kSteps = kKv == FKV_KV_BF16 ? 16 : 8;
#pragma unroll 1
    for (int c = 0; c < kSteps; ++c) {
        if (kKv == FKV_KV_FP4) {
            const uint32_t a = stage + tok * kFp4Row + 8 * c;
            if (!valid) {
                st_shared_v2_zero(a);
                if (c == 0) st_shared_v2_zero(stage + tok * kFp4Row + kFp4Codes);
            } else if ((ld_shared_u8(stage + tok * kFp4Row + kFp4Codes + c) & 0x7Fu) == 0x7Fu) {
                odd = true;                                        // codes of zero under a scale of zero
                asm volatile("st.shared.u8 [%0], %1;" ::"r"(stage + tok * kFp4Row + kFp4Codes + c), "r"(0u) : "memory");
            }
            continue;
        }
        const uint32_t a = stage + 16384 * (c >> 3) + tok * 128 + (((c & 7) ^ (tok & 7)) << 4);
        const uint4 v = ld_shared_v4(a);
        uint32_t w[4] = {v.x, v.y, v.z, v.w}, bad = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t m;                                            // the bits of what is no number
            if (kKv == FKV_KV_BF16) m = ((w[j] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((w[j] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
            else m = ((((w[j] & 0x7F7F7F7Fu) + 0x01010101u) >> 7) & 0x01010101u) * 0xFFu;
            if (!valid) m = 0xFFFFFFFFu;
            else odd |= m != 0;
            bad |= m;
            w[j] &= ~m;
        }
        if (bad) st_shared_v4(a, make_uint4(w[0], w[1], w[2], w[3]));
    }
    return odd;
}

// ---------------------------------------------------------------------------
// shares
// ---------------------------------------------------------------------------
// A block has kParts shares: k gridDim + blockIdx, so that few shares are spread over all
// blocks.  The whole block counts the tiles; where a share begins is found by the thread that
// counted the request.
template <int kThreads, int kParts>
struct TreeShares {
    int64_t scan[kThreads / 32];                                   // one per warp
    int64_t off[kParts];                                           // the share's first tile within its request
    int32_t r[kParts];                                             // that request; batch: nothing to do
};
struct TreeTotal {
    int64_t tiles, used;                                           // shares that get tiles
    __device__ __forceinline__ int64_t begin(int64_t share) const { return share < used ? tiles * share / used : tiles; }
    // The share that has tile t.
    __device__ __forceinline__ int64_t of(int64_t t) const { return ((t + 1) * used + tiles - 1) / tiles - 1; }
};
template <int kTok, int kThreads, int kParts>
__device__ __forceinline__ TreeTotal tree_shares(const TreeParams &p, int tpt, TreeShares<kThreads, kParts> &sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.batch + kThreads - 1) / kThreads;
    if (tid < kParts) sh.r[tid] = p.batch;
    TreeTotal t{0, 1};
    int64_t at = 0;
    // twice the same loop: what this thread's requests have, then where shares begin in them
    for (int pass = 0; pass < 2; ++pass) {
        int64_t mine = 0;
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int r = tid * per + i;
            if (r >= p.batch) break;
            const TreeRequest q = tree_request(p, r);
            if (!q.live) continue;
            const int64_t x = static_cast<int64_t>(tree_span<kTok>(p, q).tiles) * ((q.n + tpt - 1) / tpt) * p.hkv;
            if (pass) {
#pragma unroll 1
                for (int k = 0; k < kParts; ++k) {
                    const int64_t share = static_cast<int64_t>(k) * gridDim.x + blockIdx.x, g0 = t.begin(share);
                    if (share < t.used && g0 >= at + mine && g0 < at + mine + x) {
                        sh.r[k] = r;
                        sh.off[k] = g0 - at - mine;
                    }
                }
            }
            mine += x;
        }
        if (pass) break;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sh.scan[warp] = incl;
        __syncthreads();
        at = incl - mine;
#pragma unroll 1
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) at += sh.scan[w];
            t.tiles += sh.scan[w];
        }
        const int64_t most = static_cast<int64_t>(kParts) * gridDim.x;
        t.used = t.tiles < 1 ? 1 : t.tiles < most ? t.tiles : most;
    }
    return t;
}

// ---------------------------------------------------------------------------
// the kernels on the tensor cores' own memory (tree_attn.cu, tree_attn_wide.cu)
// ---------------------------------------------------------------------------
constexpr int kTreeTok = 128;                  // tokens of a tile
constexpr int kTreePoison = 10;                // tiles of a unit that hold tokens not seen by every row, at most (9)
constexpr uint32_t kTreeWaitTicks = 2000000000ull >> 10;      // of 1024 ns: a wait's limit
constexpr uint64_t kTreeDrainNs = 2000000000ull;

struct Ring {                                  // a buffer of a ring and the parity of its current round
    int i = 0;
    uint32_t ph = 0;
    template <int kN>
    __device__ __forceinline__ void next() {
        if (++i == kN) {
            i = 0;
            ph ^= 1;
        }
    }
};

// Waits for a phase; false: it gave up.  After `limit` ticks without it the call has failed: that
// is recorded, and from then on no wait of the block waits, so that it ends soon, with outputs
// that are not valid: a long share may have tens of thousands of waits left by then, so each
// looks at `dead` every 8 tests (one that fails has slept in hardware for 2 us).  Out of line:
// with both looks after every test 64 requests around 16k tokens, 8 drafted, took 628 us
// instead of 580 (tree_attn.cu: its roles share the instruction cache).
__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity, volatile int32_t *dead, uint32_t *err,
                                          uint32_t limit = kTreeWaitTicks) {
    if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
    uint32_t since = 0;
#pragma unroll 1
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
        if (__builtin_expect((i & 7u) == 0, 0)) {
            const uint32_t now = static_cast<uint32_t>(globaltimer_ns() >> 10);
            if (i == 8) since = now;
            if (now - since > limit) {
                *dead = 1;
                atomicOr(err, FKV_DEVERR_TIMEOUT);
            }
            if (*dead) return false;
        }
    }
    return true;
}

// ---------------------------------------------------------------------------
// rows of the cache as f16 (this thread's token)
// ---------------------------------------------------------------------------
// 64 values (half `hf`) of the row in a K or V stage, as f16 pairs.
template <int kKv>
__device__ __forceinline__ void half_row(uint32_t stage, int tok, int hf, uint32_t (&f)[32]) {
    if (kKv == FKV_KV_FP8_E4M3) {
        const uint32_t row = stage + tok * 128;
        uint4 v[4];                                                // all on their way before one is converted
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = ld_shared_v4(row + (((4 * hf + c) ^ (tok & 7)) << 4));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) e4m3x4_to_f16(w[j], f[8 * c + 2 * j], f[8 * c + 2 * j + 1]);
        }
    } else {
        const uint32_t row = stage + tok * kFp4Row;
        const uint2 sc = ld_shared_v2(row + kFp4Codes);
        const uint32_t s4 = hf ? sc.y : sc.x;
        uint2 cs[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) cs[b] = ld_shared_v2(row + 32 * hf + 8 * b);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint2 c = cs[b];
            const uint32_t s = e4m3_to_f16_pair((s4 >> (8 * b)) & 0xFFu);
            uint32_t x[4], y[4];
            e2m1x8_to_f16(c.x, x);
            e2m1x8_to_f16(c.y, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[8 * b + j] = mul_f16x2(x[j], s);
                f[8 * b + 4 + j] = mul_f16x2(y[j], s);
            }
        }
    }
}

// A row as f16 into a 128 x 128 operand buffer (two halves of 64 dims; of V MN-major, of K K-major).
template <int kKv>
__device__ __forceinline__ void convert_row(uint32_t stage, uint32_t dst, int tok) {
#pragma unroll 1
    for (int hf = 0; hf < 2; ++hf) {
        uint32_t f[32];
        half_row<kKv>(stage, tok, hf, f);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            st_shared_v4(dst + 16384 * hf + tok * 128 + ((c ^ (tok & 7)) << 4),
                         make_uint4(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3]));
    }
}

// ---------------------------------------------------------------------------
// the other parts of a call (host)
// ---------------------------------------------------------------------------
// Joins the parts of cut units (tree_attn.cu).
cudaError_t launch_tree_join(const TreeParams &p, int shares, int rows, cudaStream_t st);
// The kernel of 128 or 256 rows a unit (tree_attn_wide.cu).
constexpr int kTreeWideRows = 256;
fkv_status launch_tree_wide(const TreeParams &p, int kv, int rows, int sms, const CUtensorMap &tmK, const CUtensorMap &tmV, cudaStream_t st);
// The kernel of few rows a unit (tree_attn_small.cu): 16 or 32, FP8 or FP4.
int tree_small_shares(int sms);
constexpr int kTreeSmallTok = 32;              // its tiles' tokens
fkv_status launch_tree_small(const TreeParams &p, int kv, int rows, int sms, const CUtensorMap &tmK, const CUtensorMap &tmV, cudaStream_t st);

}  // namespace fkv
