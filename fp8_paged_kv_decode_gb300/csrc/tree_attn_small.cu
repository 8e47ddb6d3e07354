// tree_attn_small.cu -- tree and window attention of few rows: a warp for itself.
//
// Up to 32 rows a unit (a decode step over a window; small trees), FP8 or 4-bit cache: too
// few rows to pay for operands in tensor memory, and bound by memory as long as a tile's
// arithmetic stays below its share of the copy bandwidth.  So each warp streams its share's
// tiles of 32 tokens through a ring of its own and computes in registers with m16n8k16
// products, rows on M: S = Q K^T, then P, as the second product's first operand where it lies,
// O += P V.  K and V become f16 in registers on the way, once for all rows; no barrier joins
// the warps and all run the same small loop.
//
// FP8 streams at 90% of a copy's rate once it runs (a window of 4096 over 64 requests: 98 us,
// of which 10 are the start, the last tiles and the joining).  FP4 fills no unit (256 requests,
// window of 1024: 103 us, 41 at the copy's rate; issue slots 42%, DRAM 32%, tensor pipe 26%):
// a tile is 800 instructions of a warp, conversions and products for 16 rows of which a group of
// 4 uses 4, and eight warps do not cover their latencies; 12 warps of 168 registers or 16 of 128
// gained nothing (102, 126 us).
//
// Operand layouts: lane (g, t) = (lane / 4, lane % 4).
//   K of 8 tokens: token g, dims 16t .. and 64 + 16t .. (one 16-byte load each, or 8 bytes and
//   a scale), four dims a step of K; Q's fragments take the dims in the same order.
//   V of 16 tokens: tokens 2t, 2t + 1, 2t + 8, 2t + 9, dims 16g .. 16g + 15, interleaved over
//   two tokens before they are converted; product d has dims 16n + d on N, so a lane ends with
//   dims 32t .. 32t + 31 of its rows.
#include <cudaTypedefs.h>

#include <mutex>

#include "tree_attn.cuh"

namespace fkv {

constexpr int kSmallPoison = 26;               // tiles of a unit that hold tokens not seen by every row, at most

template <int kKv, int kMB>                    // kMB: blocks of 16 rows
struct SmallCfg {
    static constexpr int kRows = 16 * kMB;
    static constexpr int kRowB = kKv == FKV_KV_FP8_E4M3 ? 128 : kFp4Row;
    static constexpr int kTileB = kTreeSmallTok * kRowB, kStageB = 2 * kTileB;    // K then V
    static constexpr int kWarps = 8;
    static constexpr int kStages = kKv == FKV_KV_FP8_E4M3 ? (kMB == 1 ? 3 : 2) : (kMB == 1 ? 4 : 3);
    static constexpr int kQB = kMB == 1 ? 0 : 2 * 8 * 32 * 16;                // with 32 rows Q's fragments lie in shared memory
    static constexpr int kWarpB = kStages * kStageB + kQB;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kSmem = kWarps * kWarpB;
    static_assert(kKv != FKV_KV_FP8_E4M3 || kWarpB % 1024 == 0, "swizzled stages start on 1024 bytes");
};
template <int kKv, int kMB>
struct SmallCtrl {
    using C = SmallCfg<kKv, kMB>;
    uint64_t full[C::kWarps][C::kStages];
    uint32_t poison[C::kWarps][kSmallPoison];  // tokens whose V holds NaN, of each tile that not every row sees whole
    TreeShares<C::kThreads, C::kWarps> shares;
    int32_t dead;                              // a wait gave up
};

// 16 dims of two K chunks of token g as the second operand of the eight steps of K.
template <int kKv>
__device__ __forceinline__ void k_fragments(uint32_t tile, int row, int g, int t, uint32_t (&f)[16]) {
    if (kKv == FKV_KV_FP8_E4M3) {
        const uint4 a = ld_shared_v4(tile + row * 128 + ((t ^ g) << 4)), b = ld_shared_v4(tile + row * 128 + (((t + 4) ^ g) << 4));
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) e4m3x4_to_f16(w[j], f[2 * j], f[2 * j + 1]);
    } else {
        const uint32_t at = tile + row * kFp4Row;
        const uint2 a = ld_shared_v2(at + 8 * t), b = ld_shared_v2(at + 32 + 8 * t);
        const uint32_t s = ld_fp4_scales(at, t);                   // of blocks t and 4 + t
        const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t x[4];
            e2m1x8_to_f16(w[j], x);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[4 * j + i] = mul_f16_half(x[i], s, j >> 1);
        }
    }
}

template <int kKv, int kMB>
__global__ void __launch_bounds__(SmallCfg<kKv, kMB>::kThreads, 1)
tree_small_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = SmallCfg<kKv, kMB>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ SmallCtrl<kKv, kMB> ct;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * C::kWarpB, sQ = ring + C::kStages * C::kStageB, bars = smem_u32(ct.full[warp]);
    if (threadIdx.x == 0) ct.dead = 0;
    if (lane == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(bars + 8 * i, 1);
        fence_mbar_init();
    }
    grid_dep_wait();                                               // lengths, tables and cache of earlier kernels
    const int tpt = C::kRows / p.group;                            // tokens of a unit's rows
    const TreeTotal total = tree_shares<kTreeSmallTok, C::kThreads, C::kWarps>(p, tpt, ct.shares);
    __syncthreads();
    grid_dep_launch();

    const int share = warp * gridDim.x + blockIdx.x;
    const int64_t g1 = total.begin(share + 1);
    int64_t off = ct.shares.off[warp], left = g1 - total.begin(share);
    int r = ct.shares.r[warp];
    int4 join = make_int4(-1, 0, 0, 0);
    int stage = 0;
    uint32_t phase = 0;
    bool gone = false;                                             // a copy that did not come: nothing more is done
    while (left > 0 && r < p.batch && !gone) {
        const TreeRequest q = tree_request(p, r);
        if (!q.live) {
            ++r;
            continue;
        }
        const TreeSpan sp = tree_span<kTreeSmallTok>(p, q);
        const int mt = (q.n + tpt - 1) / tpt, units = mt * p.hkv;
        const uint64_t policy = mt > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
#pragma unroll 1
        for (int ui = static_cast<int>(off / sp.tiles), tb = static_cast<int>(off % sp.tiles); ui < units && left > 0 && !gone; ++ui, tb = 0) {
            TreeUnit u;
            u.tb = tb;
            u.te = left < sp.tiles - tb ? tb + static_cast<int>(left) : sp.tiles;
            u.h = ui / mt;
            const int m = ui - u.h * mt;
            u.tok0 = q.t0 + m * tpt;
            u.ntok = min(tpt, q.n - m * tpt);
            u.ctx = q.len - q.n;
            u.len = q.len;
            u.start = sp.start;
            u.sink_tiles = sp.sink_tiles;
            u.head = sp.head;
            u.row = q.row;
            u.slot = tb == 0 && u.te == sp.tiles ? -1 : 2 * share + (tb == 0 ? 1 : 0);
            unit_whole<kTreeSmallTok>(p, u);
            if (tb > 0 && u.te == sp.tiles)                        // the last part of a unit that other shares began
                join = make_int4(static_cast<int>(total.of(g1 - left - tb)), u.tok0, u.ntok, u.h);
            left -= u.te - u.tb;

            // ---- copies: each page's rows of a tile; page ids 32 at a time ----
            bool wrong = false;                                    // a page outside the pool
            int32_t ids = -1, ids_at = -64;                        // this lane's id of page ids_at + lane
            auto issue = [&](int i, int st) {
                const uint32_t t0 = tile_at<kTreeSmallTok>(u, i);
                const int pages = p.page_size < kTreeSmallTok && t0 + p.page_size < tile_end(u, i) ? 2 : 1;
                const int first = static_cast<int>(t0 / p.page_size), last_page = (u.len - 1) / p.page_size;
                if (first < ids_at || first + pages > ids_at + 32) {
                    ids_at = first;
                    ids = first + lane <= last_page ? __ldg(p.indices + u.row + first + lane) : -1;
                }
                const int rows = min(p.page_size, kTreeSmallTok);
                const uint32_t dst = ring + st * C::kStageB, bar = bars + 8 * st;
                if (lane == 0) mbar_arrive_expect_tx(bar, 2 * pages * rows * C::kRowB);
                __syncwarp();
#pragma unroll 1
                for (int k = 0; k < pages; ++k) {
                    int32_t pg = __shfl_sync(kAll, ids, first + k - ids_at);
                    if (static_cast<uint32_t>(pg) >= static_cast<uint32_t>(p.pages)) {
                        pg = 0;                                    // never dereferenced: the unit's rows become zeros
                        wrong = true;
                    }
                    const int at = static_cast<int>(t0 + k * p.page_size - static_cast<uint32_t>(first + k) * p.page_size);   // within the page
                    if (lane >= 2) continue;                       // lane 0: K, lane 1: V
                    const uint32_t to = dst + lane * C::kTileB + k * rows * C::kRowB;
                    if (kKv == FKV_KV_FP8_E4M3)
                        tma_load_4d(to, lane ? &tmV : &tmK, bar, 0, at, u.h, pg, policy);
                    else
                        bulk_load_hint(to, (lane ? p.v_cache : p.k_cache) + ((static_cast<int64_t>(pg) * p.hkv + u.h) * p.page_size + at) * kFp4Row,
                                       rows * kFp4Row, bar, policy);
                }
            };
            const int ahead = min(u.te - u.tb, C::kStages);
            for (int k = 0; k < ahead; ++k) issue(u.tb + k, (stage + k) % C::kStages);

            // ---- Q: f16 with a power of two per row ----
            uint32_t qa[kMB == 1 ? 8 : 1][4];
            float cs[kMB][2];                                      // a logit in log2 units per unit of S
            int tk[kMB][2];                                        // the rows' tokens (of the call)
            const float ks = __ldg(p.k_scale + u.h);
#pragma unroll
            for (int mb = 0; mb < kMB; ++mb) {
                uint32_t f[2][16];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int row = 16 * mb + g + 8 * hf, tok = row / p.group;
                    const bool there = tok < u.ntok;
                    tk[mb][hf] = there ? u.tok0 + tok : -1;
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        p.q + (static_cast<int64_t>(u.tok0 + tok) * p.hq + u.h * p.group + (row - tok * p.group)) * 128);
                    uint32_t w[16], big = 0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (there) x = __ldg(src + 2 * t + 8 * (c >> 1) + (c & 1));
                        w[4 * c] = x.x, w[4 * c + 1] = x.y, w[4 * c + 2] = x.z, w[4 * c + 3] = x.w;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) big = max(big, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
                    big = max(big, __shfl_xor_sync(kAll, big, 1));
                    big = max(big, __shfl_xor_sync(kAll, big, 2));
                    const QueryPower qp = query_power(big);
                    const float up = qp.up;
                    cs[mb][hf] = p.scale_log2 * ks * qp.down;
#pragma unroll
                    for (int j = 0; j < 16; ++j) f[hf][j] = pack_f16x2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xFFFF0000u) * up);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if constexpr (kMB == 1) {
                        qa[j][0] = f[0][2 * j], qa[j][1] = f[1][2 * j], qa[j][2] = f[0][2 * j + 1], qa[j][3] = f[1][2 * j + 1];
                    } else {
                        st_shared_v4(sQ + ((mb * 8 + j) * 32 + lane) * 16, make_uint4(f[0][2 * j], f[1][2 * j], f[0][2 * j + 1], f[1][2 * j + 1]));
                    }
                }
            }
            float o[kMB][16][4], l[kMB][2], ref[kMB][2];
#pragma unroll
            for (int mb = 0; mb < kMB; ++mb) {
                l[mb][0] = l[mb][1] = 0.f;
                ref[mb][0] = ref[mb][1] = kTreeNone;
#pragma unroll
                for (int d = 0; d < 16; ++d) o[mb][d][0] = o[mb][d][1] = o[mb][d][2] = o[mb][d][3] = 0.f;
            }
            int odd_tiles = 0;
            bool odd = false;                                      // NaN in V that not every row sees
#pragma unroll 1
            for (int i = u.tb; i < u.te; ++i) {
                const uint32_t tile = ring + stage * C::kStageB;
                if (__any_sync(kAll, !tree_wait(bars + 8 * stage, phase, &ct.dead, p.err))) {
                    gone = true;
                    break;
                }
                // ---- S = Q K^T ----
                float s[kMB][4][4];
#pragma unroll
                for (int nb = 0; nb < 4; ++nb) {
                    uint32_t f[16];
                    k_fragments<kKv>(tile, 8 * nb + g, g, t, f);
#pragma unroll
                    for (int mb = 0; mb < kMB; ++mb) {
                        s[mb][nb][0] = s[mb][nb][1] = s[mb][nb][2] = s[mb][nb][3] = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if constexpr (kMB == 1) {
                                mma_f16(s[mb][nb], qa[j][0], qa[j][1], qa[j][2], qa[j][3], f[2 * j], f[2 * j + 1]);
                            } else {
                                const uint4 a = ld_shared_v4(sQ + ((mb * 8 + j) * 32 + lane) * 16);
                                mma_f16(s[mb][nb], a.x, a.y, a.z, a.w, f[2 * j], f[2 * j + 1]);
                            }
                        }
                    }
                }
                // logits in log2 units: rounded products, as the references'
#pragma unroll
                for (int mb = 0; mb < kMB; ++mb)
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mb][nb][e] = __fmul_rn(s[mb][nb][e], cs[mb][e >> 1]);
                if (__builtin_expect(!tile_whole(u, i), 0)) {
                    const uint32_t t0 = tile_at<kTreeSmallTok>(u, i);
                    const bool bad = clean_v<kKv>(tile + C::kTileB, lane, t0 + lane < tile_end(u, i));
                    const uint32_t m32 = __ballot_sync(kAll, bad);
                    if (lane == 0) ct.poison[warp][min(odd_tiles, kSmallPoison - 1)] = m32;
                    odd |= m32 != 0;
                    ++odd_tiles;
                    const uint32_t mine = seen_of(p, u, lane < C::kRows && lane / p.group < u.ntok ? u.tok0 + lane / p.group : -1, t0, tile_end(u, i));
#pragma unroll
                    for (int mb = 0; mb < kMB; ++mb)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint32_t see = __shfl_sync(kAll, mine, 16 * mb + 8 * hf + g) >> (2 * t);
#pragma unroll
                            for (int nb = 0; nb < 4; ++nb)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (!((see >> (8 * nb + e)) & 1)) s[mb][nb][2 * hf + e] = -INFINITY;
                        }
                    fence_proxy_async_smem();                      // the stage's next copy
                    __syncwarp();
                }
                // ---- references: moved where a weight would pass f16's range ----
                float top[kMB][2];
                bool move = false;
#pragma unroll
                for (int mb = 0; mb < kMB; ++mb)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float x = fmaxf(s[mb][0][2 * hf], s[mb][0][2 * hf + 1]);
#pragma unroll
                        for (int nb = 1; nb < 4; ++nb) x = fmaxf(x, fmaxf(s[mb][nb][2 * hf], s[mb][nb][2 * hf + 1]));
                        top[mb][hf] = x;
                        move |= x - ref[mb][hf] > kTreeMost<kKv>;
                    }
                if (__builtin_expect(__any_sync(kAll, move), 0)) {
#pragma unroll
                    for (int mb = 0; mb < kMB; ++mb)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            float x = top[mb][hf];
                            x = fmaxf(x, __shfl_xor_sync(kAll, x, 1));
                            x = fmaxf(x, __shfl_xor_sync(kAll, x, 2));
                            if (x - ref[mb][hf] > kTreeMost<kKv>) {
                                const float to = tree_reference<kKv>(x), f = ex2(ref[mb][hf] - to);
                                ref[mb][hf] = to;
                                l[mb][hf] *= f;
#pragma unroll
                                for (int d = 0; d < 16; ++d) {
                                    o[mb][d][2 * hf] *= f;
                                    o[mb][d][2 * hf + 1] *= f;
                                }
                            }
                        }
                }
                // ---- weights, as the second product's first operand ----
                uint32_t pa[kMB][2][4];
#pragma unroll
                for (int mb = 0; mb < kMB; ++mb) {
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[mb][nb][e] = ex2(__fadd_rn(s[mb][nb][e], -ref[mb][e >> 1]));
                            l[mb][e >> 1] += s[mb][nb][e];
                        }
                        pa[mb][nb >> 1][2 * (nb & 1)] = pack_f16x2(s[mb][nb][0], s[mb][nb][1]);
                        pa[mb][nb >> 1][2 * (nb & 1) + 1] = pack_f16x2(s[mb][nb][2], s[mb][nb][3]);
                    }
                }
                // ---- O += P V ----
                const uint32_t tv = tile + C::kTileB;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int r0 = 16 * b + 2 * t;
                    if constexpr (kKv == FKV_KV_FP8_E4M3) {
                        const uint32_t even = tv + r0 * 128 + ((g ^ (2 * t)) << 4), odds = tv + (r0 + 1) * 128 + ((g ^ (2 * t + 1)) << 4);
                        const uint4 A = ld_shared_v4(even), B = ld_shared_v4(odds), X = ld_shared_v4(even + 1024), Y = ld_shared_v4(odds + 1024);
                        const uint32_t wa[4] = {A.x, A.y, A.z, A.w}, wb[4] = {B.x, B.y, B.z, B.w}, wx[4] = {X.x, X.y, X.z, X.w}, wy[4] = {Y.x, Y.y, Y.z, Y.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            // the same dim of tokens 2t, 2t + 1 and of 2t + 8, 2t + 9
                            uint32_t lo[4], hi[4];
                            e4m3x4_to_f16(prmt(wa[k], wb[k], 0x5140), lo[0], lo[1]);
                            e4m3x4_to_f16(prmt(wa[k], wb[k], 0x7362), lo[2], lo[3]);
                            e4m3x4_to_f16(prmt(wx[k], wy[k], 0x5140), hi[0], hi[1]);
                            e4m3x4_to_f16(prmt(wx[k], wy[k], 0x7362), hi[2], hi[3]);
#pragma unroll
                            for (int mb = 0; mb < kMB; ++mb)
#pragma unroll
                                for (int d = 0; d < 4; ++d)
                                    mma_f16(o[mb][4 * k + d], pa[mb][b][0], pa[mb][b][1], pa[mb][b][2], pa[mb][b][3], lo[d], hi[d]);
                        }
                    } else {
                        const uint32_t v0 = tv + r0 * kFp4Row, v1 = v0 + 8 * kFp4Row;
                        const Fp4Pair lo = ld_fp4_pair(v0, v0 + kFp4Row, g), hi = ld_fp4_pair(v1, v1 + kFp4Row, g);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t x[8], y[8];
                            fp4_pairs(lo, k, x);
                            fp4_pairs(hi, k, y);
#pragma unroll
                            for (int mb = 0; mb < kMB; ++mb)
#pragma unroll
                                for (int d = 0; d < 8; ++d)
                                    mma_f16(o[mb][8 * k + d], pa[mb][b][0], pa[mb][b][1], pa[mb][b][2], pa[mb][b][3], x[d], y[d]);
                        }
                    }
                }
                __syncwarp();                                      // the stage is read
                if (i + C::kStages < u.te) issue(i + C::kStages, stage);
                if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (gone) break;
            // ---- end of this share's part of the unit ----
            const bool cut = u.slot >= 0;
            const float vs = __ldg(p.v_scale + u.h);
            if (wrong && lane == 0) atomicOr(p.err, FKV_DEVERR_ATTN_PAGE);
#pragma unroll
            for (int mb = 0; mb < kMB; ++mb)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float all = l[mb][hf];
                    all += __shfl_xor_sync(kAll, all, 1);
                    all += __shfl_xor_sync(kAll, all, 2);
                    if (tk[mb][hf] < 0) continue;
                    const int row = 16 * mb + g + 8 * hf;
                    if (cut) {
                        const int64_t at = static_cast<int64_t>(u.slot) * C::kRows + row;
                        float4 *dst = reinterpret_cast<float4 *>(p.part_o + at * 128 + 32 * t);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int d = 0; d < 16; d += 4)
                                dst[4 * x + d / 4] = make_float4(o[mb][d][2 * hf + x], o[mb][d + 1][2 * hf + x], o[mb][d + 2][2 * hf + x], o[mb][d + 3][2 * hf + x]);
                        if (t == 0) p.part_ml[at] = make_float2(ref[mb][hf], wrong ? -1.f : all);
                    } else {
                        const float f = wrong || all == 0.f ? 0.f : vs / all;
                        uint4 *dst = reinterpret_cast<uint4 *>(
                            p.out + (static_cast<int64_t>(tk[mb][hf]) * p.hq + u.h * p.group + (row % p.group)) * 128 + 32 * t);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int d = 0; d < 16; d += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) w[k] = f == 0.f ? 0u : pack_bf16x2(o[mb][d + 2 * k][2 * hf + x] * f, o[mb][d + 2 * k + 1][2 * hf + x] * f);
                                dst[2 * x + d / 8] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                    }
                }
            if (__builtin_expect(odd && !wrong, 0)) {
                // NaN of V that not every row sees: left out of the product, here for those who do, in what this lane has written
                __syncwarp();
                int k = 0;
#pragma unroll 1
                for (int i = u.tb; i < u.te; ++i) {
                    if (tile_whole(u, i)) continue;
                    const uint32_t t0 = tile_at<kTreeSmallTok>(u, i), m32 = *const_cast<volatile uint32_t *>(&ct.poison[warp][min(k, kSmallPoison - 1)]);
                    ++k;
#pragma unroll 1
                    for (int j = 0; j < 32 * 2 * kMB; ++j) {
                        const int b = j & 31, hf = (j >> 5) & 1, mb = j >> 6, tok = mb ? (hf ? tk[kMB - 1][1] : tk[kMB - 1][0]) : hf ? tk[0][1] : tk[0][0];
                        if (!((m32 >> b) & 1) || tok < 0 || !sees(p, u, row_sight(p, u, tok, word_of(u, t0 + b)), t0 + b, tile_end(u, i))) continue;
                        const int row = 16 * mb + g + 8 * hf;
#pragma unroll 1
                        for (int d = 32 * t; d < 32 * t + 32; ++d) {
                            const float add = odd_value<kKv>(p, u, t0 + b, d);
                            if (add == 0.f) continue;
                            if (cut) p.part_o[(static_cast<int64_t>(u.slot) * C::kRows + row) * 128 + d] += add;
                            else p.out[(static_cast<int64_t>(tok) * p.hq + u.h * p.group + (row % p.group)) * 128 + d] = __float2bfloat16_rn(add);
                        }
                    }
                }
            }
            __syncwarp();
        }
        off = 0;
        ++r;
    }
    if (lane == 0) p.joins[share] = join;
    if (gone) {
        // copies in flight still land in this warp's memory
        const uint64_t began = globaltimer_ns();
        while (globaltimer_ns() - began < 200000000ull) __nanosleep(1000);
    }
    // ---- rows of requests without work ----
    for (int k = share; k < p.batch; k += C::kWarps * gridDim.x) {
        const TreeRequest q = tree_request(p, k);
        if (!q.rows || q.live) continue;
        uint4 *dst = reinterpret_cast<uint4 *>(p.out + static_cast<int64_t>(q.t0) * p.hq * 128);
        const int64_t words = static_cast<int64_t>(q.n) * p.hq * 16;
        for (int64_t i = lane; i < words; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {

constexpr int kMaxDev = 64;
std::mutex g_mu;
unsigned long long g_ready[kMaxDev][3][2];                         // the context in which an instance's shared memory was set

template <int kKv, int kMB>
fkv_status launch(const TreeParams &p, int sms, const CUtensorMap &tmK, const CUtensorMap &tmV, cudaStream_t st) {
    using C = SmallCfg<kKv, kMB>;
    static_assert(C::kSmem + static_cast<int>(sizeof(SmallCtrl<kKv, kMB>)) <= 232448, "shared memory of a CTA");
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return FKV_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        const unsigned long long ctx = current_context_id();
        if (ctx == 0 || g_ready[dev][kKv][kMB - 1] != ctx) {
            if (cudaFuncSetAttribute(tree_small_kernel<kKv, kMB>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
                return FKV_ERR_CUDA;
            g_ready[dev][kKv][kMB - 1] = current_context_id();
        }
    }
    if (launch_pdl(tree_small_kernel<kKv, kMB>, dim3(sms), dim3(C::kThreads), C::kSmem, st, p, tmK, tmV) != cudaSuccess) return FKV_ERR_CUDA;
    return launch_tree_join(p, sms * C::kWarps, C::kRows, st) == cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}

}  // namespace

int tree_small_shares(int sms) { return sms * SmallCfg<FKV_KV_FP8_E4M3, 1>::kWarps; }

fkv_status launch_tree_small(const TreeParams &p, int kv, int rows, int sms, const CUtensorMap &tmK, const CUtensorMap &tmV, cudaStream_t st) {
    if (kv == FKV_KV_FP8_E4M3) return rows == 16 ? launch<FKV_KV_FP8_E4M3, 1>(p, sms, tmK, tmV, st) : launch<FKV_KV_FP8_E4M3, 2>(p, sms, tmK, tmV, st);
    return rows == 16 ? launch<FKV_KV_FP4, 1>(p, sms, tmK, tmV, st) : launch<FKV_KV_FP4, 2>(p, sms, tmK, tmV, st);
}

}  // namespace fkv
