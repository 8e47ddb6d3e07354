// tree_attn_wide.cu -- tree attention of many rows (65 and more a KV head).
//
// Here the products themselves are the work, so rows go on M: S = Q K^T and O += P V, both
// 128 x 128 x 128.  A row is then a lane of tensor memory and one thread of a softmax group:
// its reference, its sum and its mask are that thread's own, no barrier or shuffle joins
// threads, and P replaces S where it lies, as the second product's operand in tensor memory.
// While one softmax group computes weights, the other's products run: with more than 128 rows
// the groups have a block of 128 rows each and share every K and V tile; with fewer they take
// one block's tiles by turns, with references and sums of their own that are joined at the end.
//
// Over BF16 weights are two words (the first truncated, the second what is left, rounded): 16
// bits of them, as one word's 8 would be the largest error of the call.  So a tile costs a block
// 24 products of 128 x 128 x 16, 80 cycles each at the rate of a large matrix product, and 16384
// exponentials, 1024 cycles of an SM.  FP8 and FP4 rows become f16 operands in shared memory, by
// four more warps; their weights are one f16 word, 16 products a tile.
//
// 16 requests of 8192 tokens, 61 drafted, 64 query heads on 8: 320 us over BF16 (475 with tokens
// on M; 140 at the rate of a large product were a weight one word, 220 as it is), 264 over FP8
// (398), 266 over FP4 (394).  What is left is a block's chain, weights after S after O, which
// two groups hide only in part.  Tried: S of half tiles, so that the softmax begins earlier, 424
// us (the tensor cores drain between products of different shapes); O of half tiles and an
// issuer that takes whichever block is ready, 386; all 128 logits of a row in registers, 348.
//
// One CTA per SM: two softmax groups of four warps, a producer (a unit's geometry; K and V tiles
// by turns into one ring), an issuer, and the four converters.
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "tree_attn.cuh"
#include "umma.cuh"

namespace fkv {

namespace wide {
constexpr int kDesc = 4;
constexpr int kQB = 32768, kStageB = 32768;                        // a block's Q; a K or V tile as an operand
constexpr int kProdW = 8, kMmaW = 9, kConvW = 10;

template <int kKv>
struct Cfg {
    static constexpr bool kConv = kKv != FKV_KV_BF16;              // K and V become f16 here
    static constexpr int kThreads = kConv ? 448 : 320;
    static constexpr int kStages = kConv ? 4 : 5;                  // of operands, K's and V's by turns
    static constexpr int kRowB = kKv == FKV_KV_FP8_E4M3 ? 128 : kKv == FKV_KV_BF16 ? 256 : kFp4Row;
    static constexpr int kRaw = !kConv ? 1 : kKv == FKV_KV_FP4 ? 3 : 2, kRawB = kConv ? kTreeTok * kRowB : 0;     // of rows as they lie in the cache
    static constexpr int kOffRing = 2 * kQB, kOffRaw = kOffRing + kStages * kStageB, kOffCtrl = kOffRaw + kRaw * kRawB;
};
template <int kKv>
struct Ctrl {
    using C = Cfg<kKv>;
    uint64_t full[C::kStages], empty[C::kStages], rfull[C::kRaw], rempty[C::kRaw];
    uint64_t qready[2], sfull[2], pready[2], odone[2], xready[2], xdone[2];
    uint64_t dfull[kDesc], dempty[kDesc], drained;
    TreeUnit unit[kDesc];
    uint32_t poison[kDesc][kTreePoison][4];                        // tokens whose V holds NaN or infinities
    TreeShares<C::kThreads, 1> shares;
    uint32_t tmem;
    int32_t dead;
};
template <int kKv>
constexpr int smem_bytes() {
    constexpr int n = Cfg<kKv>::kOffCtrl + (static_cast<int>(sizeof(Ctrl<kKv>)) + 15) / 16 * 16;
    static_assert(n <= 232448, "shared memory of a CTA");
    return n;
}

// K's and V's places in the ring they share: every other stage each.
struct Turn {
    int i;
    uint32_t ph = 0;
    template <int kStages>
    __device__ __forceinline__ void next() {
        if ((i += 2) >= kStages) {
            i -= kStages;
            ph ^= 1;
        }
    }
};

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// Two weights as two BF16 words each: the first truncated, the second what is left, rounded.
__device__ __forceinline__ void split(float a, float b, uint32_t &hi, uint32_t &lo) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    hi = prmt(x, y, 0x7632u);
    const float2 r = add2(make_float2(a, b), make_float2(__uint_as_float((x & 0xFFFF0000u) ^ 0x80000000u), __uint_as_float((y & 0xFFFF0000u) ^ 0x80000000u)));
    lo = pack_bf16x2(r.x, r.y);
}
}  // namespace wide

template <int kKv>
__global__ void __launch_bounds__(wide::Cfg<kKv>::kThreads, 1)
tree_wide_kernel(const TreeParams p, int rows, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using namespace wide;
    using C = Cfg<kKv>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctrl<kKv> &ct = *reinterpret_cast<Ctrl<kKv> *>(smem + C::kOffCtrl);
    const uint32_t sQ = smem_u32(smem), sRing = sQ + C::kOffRing, sRaw = sQ + C::kOffRaw;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile int32_t *dead = &ct.dead;
    auto bar = [&](uint64_t &b) { return smem_u32(&b); };
    auto wait = [&](uint64_t &b, uint32_t parity) { return tree_wait(smem_u32(&b), parity, dead, p.err); };
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(bar(ct.full[i]), C::kConv ? 4 : 1), mbar_init(bar(ct.empty[i]), 1);
        for (int i = 0; i < C::kRaw; ++i) mbar_init(bar(ct.rfull[i]), 1), mbar_init(bar(ct.rempty[i]), 4);
        for (int i = 0; i < 2; ++i)
            mbar_init(bar(ct.qready[i]), 4), mbar_init(bar(ct.sfull[i]), 1), mbar_init(bar(ct.pready[i]), 4), mbar_init(bar(ct.odone[i]), 1),
            mbar_init(bar(ct.xready[i]), 4), mbar_init(bar(ct.xdone[i]), 4);
        for (int i = 0; i < kDesc; ++i) mbar_init(bar(ct.dfull[i]), 1), mbar_init(bar(ct.dempty[i]), 8 + 1 + (C::kConv ? 4 : 0));
        mbar_init(bar(ct.drained), 1);
        ct.dead = 0;
        fence_mbar_init();
    }
    if (warp == kMmaW) tmem_alloc(smem_u32(&ct.tmem), 512);
    if (kKv != FKV_KV_FP4 && warp == kProdW && lane == 0) prefetch_tensormap(&tmK), prefetch_tensormap(&tmV);

    grid_dep_wait();                                               // lengths, tables and cache of earlier kernels
    const int tpt = rows / p.group;                                // tokens of a unit's rows
    const TreeTotal total = tree_shares<kTreeTok, C::kThreads, 1>(p, tpt, ct.shares);
    umma_fence_before();
    __syncthreads();
    umma_fence_after();
    const uint32_t tmem = ct.tmem;
    grid_dep_launch();

    if (warp == kProdW) {
        // ==== producer ====
        const int64_t g1 = total.begin(blockIdx.x + 1);
        int r = ct.shares.r[0];
        int64_t off = ct.shares.off[0], left = g1 - total.begin(blockIdx.x);
        int4 join = make_int4(-1, 0, 0, 0);
        Ring d;
        Turn k{0}, v{1};
        Ring raw;
        const int npg = kTreeTok / p.page_size;
        const uint64_t policy = l2_policy_evict_normal();
        for (; left > 0 && r < p.batch && !__any_sync(kAll, *dead != 0); ++r, off = 0) {
            const TreeRequest q = tree_request(p, r);
            if (!q.live) continue;
            const TreeSpan sp = tree_span<kTreeTok>(p, q);
            const int mt = (q.n + tpt - 1) / tpt, units = mt * p.hkv;
            for (int ui = static_cast<int>(off / sp.tiles), tb = static_cast<int>(off % sp.tiles); ui < units && left > 0; ++ui, tb = 0) {
                wait(ct.dempty[d.i], d.ph ^ 1);
                if (__any_sync(kAll, *dead != 0)) break;           // others may still read what is there
                TreeUnit u;
                const int m = ui % mt;
                u.tb = tb;
                u.te = left < sp.tiles - tb ? tb + static_cast<int>(left) : sp.tiles;
                u.tok0 = q.t0 + m * tpt;
                u.ntok = min(tpt, q.n - m * tpt);
                u.ctx = q.len - q.n;
                u.len = q.len;
                u.start = sp.start;
                u.sink_tiles = sp.sink_tiles;
                u.head = sp.head;
                unit_whole<kTreeTok>(p, u);
                u.row = q.row;
                u.h = ui / mt;
                u.slot = tb == 0 && u.te == sp.tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (tb == 0 ? 1 : 0);
                u.bad = u.odd = 0;
                if (lane == 0) ct.unit[d.i] = u;
                for (int i = lane; i < 4 * kTreePoison; i += 32) (&ct.poison[d.i][0][0])[i] = 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ct.dfull[d.i]));
                // the last part of a unit that other CTAs began: its first tile's CTA
                if (tb > 0 && u.te == sp.tiles) join = make_int4(static_cast<int>(total.of(g1 - left - tb)), u.tok0, u.ntok, u.h);
                auto page = [&](int i) -> int32_t {                // this lane's page of tile i; -1: none to copy
                    const uint32_t t = tile_at<kTreeTok>(u, i) + static_cast<uint32_t>(lane) * p.page_size;
                    return lane < npg && t < tile_end(u, i) ? __ldg(p.indices + u.row + t / p.page_size) : -1;
                };
                int32_t pg_next = page(tb);
                for (int i = tb; i < u.te; ++i) {
                    int32_t pg = pg_next;
                    const bool has = lane < npg && tile_at<kTreeTok>(u, i) + static_cast<uint32_t>(lane) * p.page_size < tile_end(u, i);
                    if (i + 1 < u.te) pg_next = page(i + 1);
                    if (__any_sync(kAll, has && static_cast<uint32_t>(pg) >= static_cast<uint32_t>(p.pages))) {
                        if (static_cast<uint32_t>(pg) >= static_cast<uint32_t>(p.pages)) pg = 0;   // never dereferenced: the unit's rows become zeros
                        if (lane == 0) {
                            *const_cast<volatile int32_t *>(&ct.unit[d.i].bad) = 1;
                            atomicOr(p.err, FKV_DEVERR_ATTN_PAGE);
                        }
                    }
                    const uint32_t bytes = __popc(__ballot_sync(kAll, has)) * p.page_size * C::kRowB;
                    auto copy = [&](uint64_t &full, uint32_t dst, const CUtensorMap *tm, const uint8_t *cache) {
                        if (lane == 0) mbar_arrive_expect_tx(bar(full), bytes);
                        __syncwarp();
                        if (has) {
                            if (kKv == FKV_KV_FP4) {
                                const uint32_t sz = p.page_size * kFp4Row;
                                bulk_load_hint(dst + lane * sz, cache + (static_cast<int64_t>(pg) * p.hkv + u.h) * sz, sz, bar(full), policy);
                            } else {
                                tma_load_4d(dst + lane * p.page_size * 128, tm, bar(full), 0, 0, u.h, pg, policy);
                                if (kKv == FKV_KV_BF16) tma_load_4d(dst + 16384 + lane * p.page_size * 128, tm, bar(full), 64, 0, u.h, pg, policy);
                            }
                        }
                        __syncwarp();
                    };
                    bool gone = false;                             // a wait for a stage that is still read gave up
#pragma unroll
                    for (int kv = 0; kv < 2 && !gone; ++kv) {
                        const CUtensorMap *tm = kv ? &tmV : &tmK;
                        const uint8_t *cache = kv ? p.v_cache : p.k_cache;
                        if constexpr (C::kConv) {
                            gone = __any_sync(kAll, !wait(ct.rempty[raw.i], raw.ph ^ 1));
                            if (gone) break;
                            copy(ct.rfull[raw.i], sRaw + raw.i * C::kRawB, tm, cache);
                            raw.template next<C::kRaw>();
                        } else {
                            Turn &at = kv ? v : k;
                            gone = __any_sync(kAll, !wait(ct.empty[at.i], at.ph ^ 1));
                            if (gone) break;
                            copy(ct.full[at.i], sRing + at.i * kStageB, tm, cache);
                            at.template next<C::kStages>();
                        }
                    }
                    if (gone) break;
                }
                left -= u.te - u.tb;
                d.template next<kDesc>();
            }
        }
        wait(ct.dempty[d.i], d.ph ^ 1);
        if (lane == 0 && !*dead) {
            ct.unit[d.i].te = -1;
            mbar_arrive(bar(ct.dfull[d.i]));
        }
        if (lane == 0) p.joins[blockIdx.x] = join;
        __syncwarp();
        // after a wait that gave up, the copies in flight still land in this CTA's memory
        if (*dead) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 200000000ull) __nanosleep(1000);
        }
    } else if (C::kConv && warp >= kConvW) {
        // ==== converters: rows to f16 operands, a token a thread ====
        constexpr int kF = C::kConv ? kKv : FKV_KV_FP8_E4M3;
        const int ctid = tid - 32 * kConvW;
        Ring d, raw;
        Turn k{0}, v{1};
        while (true) {
            wait(ct.dfull[d.i], d.ph);
            const TreeUnit &u = ct.unit[d.i];
            const int tb = u.tb, te = u.te;
            if (__any_sync(kAll, te < 0 || *dead)) break;
            int odd_tiles = 0;
#pragma unroll 1
            for (int i = tb; i < te; ++i) {
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    Turn &at = kv ? v : k;
                    const uint32_t src = sRaw + raw.i * C::kRawB;
                    wait(ct.rfull[raw.i], raw.ph);
                    if (__builtin_expect(kv && !tile_whole(u, i), 0)) {
                        if (clean_v<kKv>(src, ctid, tile_at<kTreeTok>(u, i) + ctid < tile_end(u, i))) {
                            atomicOr(&ct.poison[d.i][min(odd_tiles, kTreePoison - 1)][ctid >> 5], 1u << (ctid & 31));
                            *const_cast<volatile int32_t *>(&ct.unit[d.i].odd) = 1;
                        }
                        ++odd_tiles;
                    }
                    wait(ct.empty[at.i], at.ph ^ 1);
                    convert_row<kF>(src, sRing + at.i * kStageB, ctid);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(ct.full[at.i]));
                        mbar_arrive(bar(ct.rempty[raw.i]));
                    }
                    at.template next<C::kStages>();
                    raw.template next<C::kRaw>();
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(ct.dempty[d.i]));
            d.template next<kDesc>();
        }
        __syncwarp();
    } else if (warp == kMmaW) {
        // ==== issuer ====
        constexpr uint32_t kHi = umma_desc_hi(1024);
        constexpr uint32_t idS = umma_idesc(!C::kConv, false, false, 128, 128), idO = umma_idesc(!C::kConv, false, true, 128, 128);
        constexpr int kO = C::kConv ? 8 : 16;                      // products of O: 16 tokens of a word each
        const uint32_t lQ = umma_desc_lo(sQ, 16), lK = umma_desc_lo(sRing, 16), lV = umma_desc_lo(sRing, 16384);
        Ring d;
        Turn k{0}, v{1};
        uint32_t nq = 0, np = 0, any = 0;                          // bit g: parity of block g's units and tiles so far; had tiles
        auto put_s = [&](int g, int q, bool last) {                // S of stage k.i with Q block q
            if ((any >> g) & 1) wait(ct.odone[g], ((np >> g) & 1) ^ 1);    // it takes the place of the weights that O was made of
            umma_fence_after();
            __syncwarp();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t at = (kk >> 2) * 1024 + (kk & 3) * 2;
                    umma_ss(tmem + 128 * g, umma_desc(lQ + q * (kQB / 16) + at, kHi), umma_desc(lK + k.i * (kStageB / 16) + at, kHi), idS, kk > 0);
                }
                umma_commit(bar(ct.sfull[g]));
                if (last) umma_commit(bar(ct.empty[k.i]));
            }
            __syncwarp();
        };
        auto put_o = [&](int g, bool add, bool last) {             // O of stage v.i
            wait(ct.pready[g], (np >> g) & 1);
            np ^= 1u << g;
            any |= 1u << g;
            umma_fence_after();
            __syncwarp();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kO; ++kk) {
                    // half a tile's weights: 32 columns a word, from column 0 or 64
                    const int half = kk / (kO / 2), word = C::kConv ? 0 : (kk >> 2) & 1, step = kk & 3;
                    umma_ts(tmem + 256 + 128 * g, tmem + 128 * g + 64 * half + 32 * word + 8 * step,
                            umma_desc(lV + v.i * (kStageB / 16) + (4 * half + step) * 128, kHi), idO, add || kk > 0);
                }
                umma_commit(bar(ct.odone[g]));
                if (last) umma_commit(bar(ct.empty[v.i]));
            }
            __syncwarp();
        };
        auto q_there = [&](int g) {
            wait(ct.qready[g], (nq >> g) & 1);
            nq ^= 1u << g;
        };
        while (true) {
            wait(ct.dfull[d.i], d.ph);
            const int tb = *const_cast<volatile int32_t *>(&ct.unit[d.i].tb), te = *const_cast<volatile int32_t *>(&ct.unit[d.i].te);
            const int blocks = *const_cast<volatile int32_t *>(&ct.unit[d.i].ntok) * p.group > 128 ? 2 : 1;
            if (__any_sync(kAll, te < 0 || *dead)) break;
            if (elect_one()) mbar_arrive(bar(ct.dempty[d.i]));
            d.template next<kDesc>();
            // S runs ahead of O by a tile of each softmax group
            const int ahead = 3 - blocks;
#pragma unroll 1
            for (int j = 0; j < te - tb + ahead; ++j) {
                const bool o = j >= ahead, sn = j < te - tb;
                if (o) wait(ct.full[v.i], v.ph);
                if (blocks == 2) {
                    // O of a tile, then S of the next one, block after block
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (o) put_o(g, j > 1, g == 1);
                        if (sn) {
                            if (j == 0) q_there(g);
                            if (g == 0) wait(ct.full[k.i], k.ph);
                            put_s(g, g, g == 1);
                        }
                    }
                } else {
                    // one block: its tiles by turns to the softmax groups
                    if (o) put_o(j & 1, j > 3, true);
                    if (sn) {
                        if (j == 0) q_there(0);
                        wait(ct.full[k.i], k.ph);
                        put_s(j & 1, 0, true);
                    }
                }
                if (o) v.template next<C::kStages>();
                if (sn) k.template next<C::kStages>();
            }
        }
        __syncwarp();
        if (elect_one()) umma_commit(bar(ct.drained));             // nothing is in flight when the block ends
        __syncwarp();
        mbar_wait_bounded(bar(ct.drained), 0, kTreeDrainNs);
    } else {
        // ==== softmax ====
        const int g = warp >> 2, gtid = tid & 127;
        const uint32_t tlane = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + tlane + 128 * g, tO = tmem + tlane + 256 + 128 * g;
        float c = p.scale_log2, c_next = c;                        // a logit in log2 units per unit of S
        Ring d;
        Turn v{1};
        uint32_t n = 0, n_other = 0, n_turns = 0;                  // tiles of this group and the other, units in turns so far
        auto load_q = [&](const TreeUnit &u) {
            // the warp's own rows, two at a time; f16 with a power of two per row (BF16: as it is)
            const bool alone = u.ntok * p.group <= 128;            // one block, which group 0 loads
            const int c16 = lane & 15, row0 = (alone ? 0 : 128 * g) + 32 * (warp & 3) + (lane >> 4);
            const float ks = C::kConv ? __ldg(p.k_scale + u.h) : 1.f;
#pragma unroll 1
            for (int r8 = 0; r8 < 16; r8 += 8) {
                uint4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int rr = row0 + 2 * (r8 + i), tk = rr / p.group;
                    x[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (tk < u.ntok)
                        x[i] = __ldg(reinterpret_cast<const uint4 *>(
                                         p.q + (static_cast<int64_t>(u.tok0 + tk) * p.hq + u.h * p.group + (rr - tk * p.group)) * 128) + c16);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int rr = (row0 & 127) + 2 * (r8 + i);
                    if constexpr (C::kConv) {
                        uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, big = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) big = max(big, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
#pragma unroll
                        for (int o = 1; o < 16; o <<= 1) big = max(big, __shfl_xor_sync(kAll, big, o));
                        const QueryPower qp = query_power(big);
                        // (the scale's sign goes to Q, and a factor of zero, or one that underflows, is next to nothing: |S| is
                        // below 2^36, so its logits are zero all the same, and -infinity times it is itself)
                        const float up = copysignf(qp.up, ks);
                        const float down = __shfl_sync(kAll, qp.down, 16 * (lane & 1));
                        const float cr = p.scale_log2 * fabsf(ks) * down;
                        if (lane >> 1 == r8 + i) c_next = cr < 0x1p-126f ? 0x1p-126f : cr;     // (NaN stays)
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = pack_f16x2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xFFFF0000u) * up);
                        x[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (!alone || g == 0) st_shared_v4(sQ + g * kQB + (c16 >> 3) * 16384 + rr * 128 + (((c16 & 7) ^ (rr & 7)) << 4), x[i]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && (!alone || g == 0)) mbar_arrive(bar(ct.qready[g]));
        };
        wait(ct.dfull[0], 0);
        if (!__any_sync(kAll, *dead || ct.unit[0].te < 0)) load_q(ct.unit[0]);
        while (true) {
            const TreeUnit &u = ct.unit[d.i];
            const int tb = u.tb, te = u.te;
            if (__any_sync(kAll, te < 0 || *dead)) break;
            const bool turns = u.ntok * p.group <= 128;            // one block: its tiles by turns
            const int row = turns ? gtid : 128 * g + gtid, rtok = row / p.group, rhead = row - rtok * p.group;
            const int tok = rtok < u.ntok ? u.tok0 + rtok : -1;    // the row's token (of the call)
            float ref = kTreeNone, l = 0.f;
            bool far = false;                                      // of any of the warp's rows: products are rounded first
            int odd_tiles = 0;
            c = c_next;
#pragma unroll 1
            for (int i = tb; i < te; ++i) {
                if (turns && ((i - tb - g) & 1)) {
                    odd_tiles += !tile_whole(u, i);
                    if (!C::kConv) v.template next<C::kStages>();
                    continue;
                }
                wait(ct.sfull[g], n & 1);
                umma_fence_after();
                // 64 logits at a time, their weights' two words in their place
                const bool whole = tile_whole(u, i);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                // (two forms of the loop: a branch in each half costs trees of 61 over FP8 272 us instead of 264)
                auto weights = [&](auto rounded, int at) {         // from token `at` on; returns where references got far
                    constexpr bool kRounded = decltype(rounded)::value;
#pragma unroll 1
                    for (; at < 128; at += 64) {
                        float s[64];
                        tmem_load(tS + at, s);
                        if (__builtin_expect(!whole, 0)) {
                            const uint32_t t0 = tile_at<kTreeTok>(u, i) + at;
                            const uint32_t end = tile_end(u, i);
                            const uint64_t see = seen_of(p, u, tok, t0, end) | static_cast<uint64_t>(seen_of(p, u, tok, t0 + 32, end)) << 32;
#pragma unroll
                            for (int j = 0; j < 64; ++j)
                                if (!((see >> j) & 1)) s[j] = -INFINITY;   // (c is above zero)
                        }
                        float top = -INFINITY;
#pragma unroll
                        for (int j = 0; j < 64; j += 2) top = fmaxf(top, fmaxf(s[j], s[j + 1]));
                        top = __fmul_rn(top, c);
                        const bool move = __fsub_rn(top, ref) > kTreeMost<kKv>;
                        if (__builtin_expect(__any_sync(kAll, move), 0)) {
                            // the sums so far, and the weights of the tile's first half, are scaled to the new reference
                            const float to = move ? tree_reference<kKv>(top) : ref, f = move ? ex2(ref - to) : 1.f;
                            if (i > tb + turns) {
                                wait(ct.odone[g], (n - 1) & 1);
                                umma_fence_after();
#pragma unroll 1
                                for (int b = 0; b < 128; b += 32) {
                                    float o[32];
                                    uint32_t w[32];
                                    tmem_load(tO + b, o);
#pragma unroll
                                    for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(move ? o[j] * f : o[j]);
                                    tmem_store(tO + b, w);
                                }
                            }
                            if (at) {
                                tmem_store_wait();
#pragma unroll 1
                                for (int b = 0; b < 32; b += 8) {
                                    float hi[8];
                                    uint32_t wh[8];
                                    tmem_load(tS + b, hi);
                                    if constexpr (C::kConv) {
#pragma unroll
                                        for (int j = 0; j < 8; ++j) {
                                            const uint32_t x = __float_as_uint(hi[j]);
                                            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&x));
                                            wh[j] = pack_f16x2(y.x * f, y.y * f);
                                        }
                                    } else {
                                        float lo[8];
                                        uint32_t wl[8];
                                        tmem_load(tS + 32 + b, lo);
#pragma unroll
                                        for (int j = 0; j < 8; ++j) {
                                            const uint32_t x = __float_as_uint(hi[j]), y = __float_as_uint(lo[j]);
                                            split((__uint_as_float(x << 16) + __uint_as_float(y << 16)) * f,
                                                  (__uint_as_float(x & 0xFFFF0000u) + __uint_as_float(y & 0xFFFF0000u)) * f, wh[j], wl[j]);
                                        }
                                        tmem_store(tS + 32 + b, wl);
                                    }
                                    tmem_store(tS + b, wh);
                                }
                            }
                            l *= f;
                            sum[0].x *= f, sum[0].y *= f, sum[1].x *= f, sum[1].y *= f;
                            ref = to;
                            far = __any_sync(kAll, reference_far(ref));
                            if (!kRounded && far) return at;           // once more, with what is scaled already
                        }
                        const float2 c2 = make_float2(c, c), r2 = make_float2(-ref, -ref);
                        uint32_t hi[32];
                        [[maybe_unused]] uint32_t lo[C::kConv ? 1 : 32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            float2 x;
                            if constexpr (kRounded) x = make_float2(__fadd_rn(__fmul_rn(s[2 * j], c), -ref), __fadd_rn(__fmul_rn(s[2 * j + 1], c), -ref));
                            else x = fma2(make_float2(s[2 * j], s[2 * j + 1]), c2, r2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            sum[j & 1] = add2(sum[j & 1], x);
                            if constexpr (C::kConv) hi[j] = pack_f16x2(x.x, x.y);
                            else split(x.x, x.y, hi[j], lo[j]);
                        }
                        tmem_store(tS + at, hi);
                        if constexpr (!C::kConv) tmem_store(tS + at + 32, lo);
                    }
                    return at;
                };
                const int got = far ? 0 : weights(std::false_type{}, 0);
                if (__builtin_expect(got < 128, 0)) weights(std::true_type{}, got);
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                if (__builtin_expect(!C::kConv && !whole, 0)) {
                    if (g == 0 || turns) {                         // of two blocks both products with V come after block 0's weights
                        wait(ct.full[v.i], v.ph);
                        if (clean_v<kKv>(sRing + v.i * kStageB, gtid, tile_at<kTreeTok>(u, i) + gtid < tile_end(u, i))) {
                            atomicOr(&ct.poison[d.i][min(odd_tiles, kTreePoison - 1)][gtid >> 5], 1u << (gtid & 31));
                            *const_cast<volatile int32_t *>(&ct.unit[d.i].odd) = 1;
                        }
                        fence_proxy_async_smem();
                    }
                    ++odd_tiles;
                }
                tmem_store_wait();
                umma_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ct.pready[g]));
                ++n;
                if (!C::kConv) v.template next<C::kStages>();
            }
            const int mine = turns ? (te - tb + 1 - g) / 2 : te - tb, others = turns ? (te - tb + g) / 2 : te - tb;
            n_other += others;
            Ring e = d;
            e.template next<kDesc>();
            auto next_q = [&] {
                wait(ct.dfull[e.i], e.ph);
                if (!__any_sync(kAll, *dead || *const_cast<volatile int32_t *>(&ct.unit[e.i].te) < 0)) load_q(ct.unit[e.i]);
            };
            if (!turns) next_q();                                  // while the last products run
            {
                if (mine) wait(ct.odone[g], (n - 1) & 1);
                float f = 1.f, f_other = 0.f;                      // of this group's sums and the other's
                if (turns) {
                    // one row is this thread's and the other group's; Q's second block lends the room
                    float2 *x = reinterpret_cast<float2 *>(smem + kQB);
                    if (others) wait(ct.odone[g ^ 1], (n_other - 1) & 1);
                    x[128 * g + gtid] = make_float2(ref, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(ct.xready[g]));
                    wait(ct.xready[g ^ 1], n_turns & 1);
                    const volatile float2 *theirs = x + 128 * (g ^ 1) + gtid;
                    const float2 y = make_float2(theirs->x, theirs->y);
                    const float top = l == 0.f ? y.x : y.y == 0.f ? ref : fmaxf(ref, y.x);
                    f = l == 0.f ? 0.f : ex2(ref - top);
                    f_other = y.y == 0.f ? 0.f : ex2(y.x - top);
                    // (the same sum in both groups)
                    l = g ? f_other * y.y + f * l : f * l + f_other * y.y;
                    ref = top;
                }
                umma_fence_after();
                const bool wrong = *const_cast<volatile int32_t *>(&ct.unit[d.i].bad) != 0, cut = u.slot >= 0;
                const int64_t at = static_cast<int64_t>(u.slot) * rows + row;
                const int d0 = turns ? 64 * g : 0, d1 = turns ? d0 + 64 : 128;     // the dims that this thread writes
                __nv_bfloat16 *const out = p.out + (static_cast<int64_t>(tok) * p.hq + u.h * p.group + rhead) * 128;
                if (cut) {
                    if (tok >= 0 && d0 == 0) p.part_ml[at] = make_float2(ref, wrong ? -1.f : l);
                } else {
                    const float norm = wrong || l == 0.f ? 0.f : (C::kConv ? __ldg(p.v_scale + u.h) : 1.f) / l;
                    f *= norm;
                    f_other *= norm;
                }
#pragma unroll 1
                for (int b = d0; b < d1; b += 32) {
                    float o[32];
                    tmem_load(tO + b, o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = f == 0.f ? 0.f : o[j] * f;
                    if (turns) {
                        float z[32];
                        tmem_load(tmem + tlane + 256 + 128 * (g ^ 1) + b, z);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] += f_other == 0.f ? 0.f : z[j] * f_other;
                    }
                    if (tok < 0) continue;
                    if (cut) {
                        float4 *dst = reinterpret_cast<float4 *>(p.part_o + at * 128 + b);
#pragma unroll
                        for (int j = 0; j < 8; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(out + b);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) w[x] = pack_bf16x2(o[8 * j + 2 * x], o[8 * j + 2 * x + 1]);
                            dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                umma_fence_before();
                if (__builtin_expect(*const_cast<volatile int32_t *>(&ct.unit[d.i].odd) && !wrong && tok >= 0, 0)) {
                    // NaN and infinities of V that not every row sees: left out of the product, here for those who do
                    int k = 0;
#pragma unroll 1
                    for (int i = tb; i < te; ++i) {
                        if (tile_whole(u, i)) continue;
                        const uint32_t t0 = tile_at<kTreeTok>(u, i);
#pragma unroll 1
                        for (int b = 0; b < kTreeTok; ++b) {
                            if (!((*const_cast<volatile uint32_t *>(&ct.poison[d.i][min(k, kTreePoison - 1)][b >> 5]) >> (b & 31)) & 1)) continue;
                            if (!sees(p, u, row_sight(p, u, tok, word_of(u, t0 + b)), t0 + b, tile_end(u, i))) continue;
#pragma unroll 1
                            for (int dim = d0; dim < d1; ++dim) {
                                const float add = odd_value<kKv>(p, u, t0 + b, dim);
                                if (add == 0.f) continue;
                                if (cut) p.part_o[at * 128 + dim] += add;
                                else out[dim] = __float2bfloat16_rn(__bfloat162float(out[dim]) + add);
                            }
                        }
                        ++k;
                    }
                }
            }
            __syncwarp();
            if (turns) {
                // all eight warps have read the sums: the next unit's Q may lie over those that this group's other warps
                // read, and its sums over the other group's
                if (lane == 0) mbar_arrive(bar(ct.xdone[g]));
                wait(ct.xdone[0], n_turns & 1);
                wait(ct.xdone[1], n_turns & 1);
                ++n_turns;
                next_q();
            }
            if (lane == 0) mbar_arrive(bar(ct.dempty[d.i]));
            d = e;
        }
        // ---- rows of requests without work ----
        __syncwarp();
        for (int r = blockIdx.x; r < p.batch; r += gridDim.x) {
            const TreeRequest q = tree_request(p, r);
            if (!q.rows || q.live) continue;
            uint4 *o = reinterpret_cast<uint4 *>(p.out + static_cast<int64_t>(q.t0) * p.hq * 128);
            const int64_t words = static_cast<int64_t>(q.n) * p.hq * 16;
            for (int64_t i = tid; i < words; i += 256) o[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
    }
    umma_fence_before();
    __syncthreads();
    if (warp == kMmaW) {
        umma_fence_after();
        tmem_free(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {
constexpr int kMaxDev = 64;
std::mutex g_mu;
unsigned long long g_ready[kMaxDev][3];                            // the context in which an instance's shared memory was set

template <int kKv>
fkv_status launch(const TreeParams &p, int rows, int sms, const CUtensorMap &tmK, const CUtensorMap &tmV, cudaStream_t st) {
    constexpr int smem = wide::smem_bytes<kKv>();
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return FKV_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        const unsigned long long ctx = current_context_id();
        if (ctx == 0 || g_ready[dev][kKv] != ctx) {
            if (cudaFuncSetAttribute(tree_wide_kernel<kKv>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return FKV_ERR_CUDA;
            g_ready[dev][kKv] = current_context_id();
        }
    }
    if (launch_pdl(tree_wide_kernel<kKv>, dim3(sms), dim3(wide::Cfg<kKv>::kThreads), smem, st, p, rows, tmK, tmV) != cudaSuccess)
        return FKV_ERR_CUDA;
    return launch_tree_join(p, sms, rows, st) == cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}
}  // namespace

fkv_status launch_tree_wide(const TreeParams &p, int kv, int rows, int sms, const CUtensorMap &tmK, const CUtensorMap &tmV, cudaStream_t st) {
    return kv == FKV_KV_BF16         ? launch<FKV_KV_BF16>(p, rows, sms, tmK, tmV, st)
           : kv == FKV_KV_FP8_E4M3 ? launch<FKV_KV_FP8_E4M3>(p, rows, sms, tmK, tmV, st)
                                   : launch<FKV_KV_FP4>(p, rows, sms, tmK, tmV, st);
}

}  // namespace fkv
