// tree_attn.cu -- attention of drafted tokens, and over a window, on the paged cache.
//
// Request r has n drafted tokens, the last n of its seq_lens[r] cached ones.  Each is
// a query row (per query head) that sees the committed tokens before them (all of
// them, or those of a window and a few first ones) and the drafted tokens its mask names:
//     out[i][hq] = sum_t softmax_t(sm_scale * q[i][hq] . k_t) v_t   over t seen by i
// A decode step over a window is the same with one token a request.
//
// The n drafted tokens of a request and the G query heads of a KV head share its K and V,
// so a unit of work is (request, KV head, up to kR of their n G rows).  Three kernels, by the
// rows that G times the call's mean n come to, so that few rows cost little and K and V pass
// through once for all of them:
//   here               BF16 up to 64 rows, FP8 and FP4 33 to 64: products of 128-token tiles
//                      with kR = 16, 32 or 64 columns, on the fifth-generation tensor
//                      cores, tokens (or dims) on M and rows on N,
//                          S^T = K Q^T  [128 tokens][kR],   O^T = V^T P^T  [128 dims][kR]
//   tree_attn_small.cu FP8 and FP4 up to 32 rows
//   tree_attn_wide.cu  more
//
// One CTA per SM takes an equal share of all units' tiles (a unit may be cut; its parts are
// joined by a second kernel).  Its warps:
//   producer   a unit's geometry, and TMA copies of its pages into rings of K and V stages
//   converters (FP8, FP4) K and V rows to f16 in tensor memory; a unit's Q as f16, scaled by
//              one power of two (BF16: as it is)
//   issuers    a warp for S, one for O
//   softmax    two groups of four warps, one token a thread: weights against a running
//              reference, stored as the second product's operand.  The groups take turns at
//              tiles, with references and sums of their own that are joined at a unit's end
// The reference of a column moves only when a weight would pass its range: a maximum is
// put at 2^10, later ones may grow to 2^15.9 (BF16: 2^-6 and 1), so sums are rescaled a few
// times per unit.
// FP8 and FP4 weights are one f16 word, BF16 ones two BF16 words.
//
// Few rows over BF16 are bound by memory (8 requests, window of 32768: 86 us, 93% of a copy's
// rate).  64 requests around 16k tokens, 8 drafted, over FP8 take 422 to 482 us a million tokens
// (302 at a copy's rate), by their lengths; FP4 870 to 960 us in all, BF16 905: a tile's way
// through five kinds of warps, and the instruction cache that their code shares, cost what is
// missing.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <mutex>
#include <type_traits>

#include "tree_attn.cuh"
#include "umma.cuh"

namespace fkv {

// ---------------------------------------------------------------------------
// shared memory
// ---------------------------------------------------------------------------
template <int kKv, int kR>
struct TreeCfg {
    static constexpr bool kConv = kKv != FKV_KV_BF16;              // K and V become f16 here
    static constexpr int kRowB = kKv == FKV_KV_FP8_E4M3 ? 128 : kKv == FKV_KV_BF16 ? 256 : kFp4Row;
    static constexpr int kStageB = kTreeTok * kRowB;               // the K (or V) rows of a tile
    static constexpr int kNK = kKv == FKV_KV_FP4 ? 8 : kConv ? 5 : 2;
    static constexpr int kNV = kKv == FKV_KV_FP4 ? 8 : kConv ? 5 : kR <= 32 ? 3 : 2;
    static constexpr int kParts = kConv ? 1 : 2;                   // words of a weight
    static constexpr int kPW = kR <= 32 ? 64 : 16384;              // from a weight's first word to its second
    static constexpr int kPB = kR <= 32 ? 16384 : kParts * kPW;    // a weight buffer
    static constexpr int kQB = kR * 256;
    static_assert(kR <= 64 && (!kConv || kR == 64), "fewer rows of FP8 and FP4: tree_attn_small.cu; more: tree_attn_wide.cu");
    // Softmax warps with many columns take registers of the others: of a thread, at launch, then
    // of the three kinds of warps (no more in all than at launch; whole groups of four warps).
    static constexpr bool kShift = kR >= 32;
    static constexpr int kThreads = 512;                           // softmax 256, converters 128; producer, two issuers, an idle warp
    static constexpr int kRegs = 128;
    static constexpr int kRegsSoft = kR >= 64 ? 176 : 152, kRegsConv = kR >= 64 ? 88 : 104, kRegsRest = kR >= 64 ? 72 : 104;
    static_assert(2 * kRegsSoft + kRegsConv + kRegsRest <= kThreads / 128 * kRegs, "the block's registers");
    static constexpr int kND = 4;                                  // units in flight
    // tensor memory columns: K f16 (two buffers), V f16 (two), S and O (one per softmax group)
    static constexpr int kTmV = 128, kTmS = kConv ? 256 : 0, kTmO = kTmS + 2 * kR;
    static_assert(kTmO + 2 * kR <= 512, "tensor memory");
    static constexpr int kNVR = kConv ? 2 : kNV;                   // buffers between converters and issuer
    static constexpr int kOffP = kQB, kOffK = kOffP + 2 * kPB;
    static constexpr int kOffV = kOffK + kNK * kStageB, kOffCtrl = kOffV + kNV * kStageB;
};

template <int kKv, int kR>
struct TreeCtrl {
    using C = TreeCfg<kKv, kR>;
    uint64_t kfull[C::kNK], kempty[C::kNK], vfull[C::kNV], vempty[C::kNV];
    uint64_t k16full[2], k16empty[2], vready[C::kNVR], v16empty[2];
    uint64_t sfull[2], sempty[2], pfull[2], pempty[2];
    uint64_t qfull, qempty, oempty, drained[2];
    uint64_t dfull[C::kND], dempty[C::kND], cfull[C::kND];
    TreeUnit unit[C::kND];
    float colscale[C::kND];                                        // a logit in log2 units per unit of S
    uint32_t qmax[C::kND];                                         // the largest |q| of the unit, as bf16 bits
    // [unit's parity][group]: the columns' references, negated, and their warps' sums (or maxima);
    // a moved reference's factor; the factors of the two groups' sums
    alignas(16) float ref[2][2][kR];
    alignas(16) float red[2][2][4][kR];
    alignas(16) float up[2][kR];
    alignas(16) float2 part[kR];
    uint32_t poison[C::kND][kTreePoison][4];                       // tokens whose V holds NaN or infinities
    TreeShares<C::kThreads, 1> shares;
    uint32_t tmem;
    int32_t dead;
};

template <int kKv, int kR>
constexpr int tree_smem() {
    using C = TreeCfg<kKv, kR>;
    using T = TreeCtrl<kKv, kR>;
    static_assert(offsetof(T, ref) % 16 == 0 && offsetof(T, up) % 16 == 0 && offsetof(T, part) % 16 == 0 && C::kOffCtrl % 16 == 0, "read four at a time");
    static_assert(C::kOffP % 1024 == 0 && C::kOffK % 1024 == 0 && C::kOffV % 1024 == 0,
                  "swizzled buffers start on 1024 bytes");
    return TreeCfg<kKv, kR>::kOffCtrl + static_cast<int>((sizeof(TreeCtrl<kKv, kR>) + 15) / 16 * 16);
}

// Whether any of the 128 threads of a softmax group says so (a barrier of the group).
__device__ __forceinline__ bool group_any(int id, bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(x ? 1u : 0u), "r"(id) : "memory");
    return r != 0;
}
__device__ __forceinline__ bool both_any(bool x) {             // the same for both groups
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 3, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(x ? 1u : 0u) : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }

__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}

// Bits of this group's columns whose rows see token t of a tile up to `end` (rows past the unit's: unset).
template <int kNC>
__device__ __forceinline__ uint64_t seen_by(const TreeParams &p, const TreeUnit &u, int col0, uint32_t t, uint32_t end) {
    uint64_t v = 0;
    const int w = word_of(u, t), G = p.group;
    for (int i = col0 / G; i < u.ntok && i * G < col0 + kNC; ++i) {
        if (sees(p, u, row_sight(p, u, u.tok0 + i, w), t, end)) {
            const int a = max(i * G, col0) - col0, b = min((i + 1) * G, col0 + kNC) - col0;
            v |= (b - a == 64 ? ~0ull : (1ull << (b - a)) - 1) << a;
        }
    }
    return v;
}

// ---------------------------------------------------------------------------
// V as f16 in tensor memory
// ---------------------------------------------------------------------------
// The V rows of a stage as f16 into tensor memory: dims on lanes, two tokens a column, from
// column `dst` (of this warp's 32 lanes, dims 32 cw ..).  Thread l holds, of tokens 8k + 2 (l % 4)
// and the next one, the places of the .16x128b store: register 2k of the lower (upper) 16 lanes
// is lane l / 4, register 2k + 1 lane 8 + l / 4.  The two tokens' codes are interleaved before
// they are converted, so that a converted pair is one dim of both.
// FP8: a transposing load brings two dims of both tokens; lane 16b + 8h + r is dim 16b + 2r + h.
// FP4: rows of 72 bytes cannot be loaded so (every other one starts in the middle of 16
// bytes): two bytes a token, four dims; lane 16b + 8h + r is dim 4r + 2b + h.
template <int kKv>
__device__ __forceinline__ void convert_v_tmem(uint32_t stage, uint32_t dst, int cw, int lane) {
    if constexpr (kKv == FKV_KV_FP8_E4M3) {
        const uint32_t row = stage + lane * 128;                   // of 32 tokens at a time
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
            uint32_t in[2][8];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint32_t at = row + hf * 8192 + (((2 * cw + b) ^ (lane & 7)) << 4);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(in[b][4 * q]), "=r"(in[b][4 * q + 1]), "=r"(in[b][4 * q + 2]), "=r"(in[b][4 * q + 3])
                                 : "r"(at + q * 4096));
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t f[16];
#pragma unroll
                for (int k = 0; k < 8; ++k) e4m3x4_to_f16(prmt(in[b][k], 0u, 0x3120u), f[2 * k], f[2 * k + 1]);
                tmem_store_rows(dst + (static_cast<uint32_t>(16 * b) << 16) + 32 * hf, f);
            }
        }
        return;
    }
    const int g = lane >> 2, t = lane & 3;
    const uint32_t r0 = stage + 2 * t * kFp4Row + 16 * cw + 2 * g, s0 = stage + 2 * t * kFp4Row + kFp4Codes + 2 * cw + (g >> 2);
#pragma unroll 1
    for (int hf = 0; hf < 2; ++hf) {
        uint32_t a[16], b[16], in[8][2], sin[8][2];                // all loads on their way before one word is converted
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                in[k][j] = ld_shared_u16(r0 + (64 * hf + 8 * k + j) * kFp4Row);
                sin[k][j] = ld_shared_u8(s0 + (64 * hf + 8 * k + j) * kFp4Row);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            // byte 0: dim 0 of both tokens, byte 1: dim 2; and dims 1 and 3
            const uint32_t w0 = in[k][0], w1 = in[k][1];
            const uint32_t even = (w0 & 0x0F0Fu) | ((w1 << 4) & 0xF0F0u), odd = ((w0 >> 4) & 0x0F0Fu) | (w1 & 0xF0F0u);
            uint32_t f[4];
            e2m1x8_to_f16(even | (odd << 16), f);
            const uint32_t s = e4m3x2_to_f16x2(static_cast<uint16_t>(sin[k][0] | (sin[k][1] << 8)));
            a[2 * k] = mul_f16x2(f[0], s);
            a[2 * k + 1] = mul_f16x2(f[2], s);
            b[2 * k] = mul_f16x2(f[1], s);
            b[2 * k + 1] = mul_f16x2(f[3], s);
        }
        tmem_store_rows(dst + 32 * hf, a);
        tmem_store_rows(dst + (16u << 16) + 32 * hf, b);
    }
}
// The dim of a lane of O (within its warp's 32).
template <int kKv>
__device__ __forceinline__ int dim_of_lane(int lane) {
    if (kKv == FKV_KV_BF16) return lane;
    const int b = lane >> 4, h = (lane >> 3) & 1, r = lane & 7;
    return kKv == FKV_KV_FP8_E4M3 ? 16 * b + 2 * r + h : 4 * r + 2 * b + h;
}

// kN columns reduced over a warp's lanes: half of them go to the lane kO away, then half of
// those that are left, and so on; at the end a lane has kN / 32 columns (at least one).
template <int kN, int kO, int kSize, typename Op>
__device__ __forceinline__ void spread(float (&v)[kSize], int lane, Op op) {
    if constexpr (kO > 0) {
        constexpr int n = kN > 1 ? kN / 2 : 1;
        if constexpr (kN > 1) {
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const float a = v[j], b = v[j + n];
                v[j] = op(lane & kO ? b : a, __shfl_xor_sync(kAll, lane & kO ? a : b, kO));
            }
        } else {
            v[0] = op(v[0], __shfl_xor_sync(kAll, v[0], kO));
        }
        spread<n, kO / 2>(v, lane, op);
    }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int kKv, int kR>
__global__ void __launch_bounds__(TreeCfg<kKv, kR>::kThreads, 1)
tree_attn_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = TreeCfg<kKv, kR>;
    using Ctrl = TreeCtrl<kKv, kR>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctrl &ct = *reinterpret_cast<Ctrl *>(smem + C::kOffCtrl);
    const uint32_t base = smem_u32(smem);
    const uint32_t sQ = base, sP = base + C::kOffP, sK = base + C::kOffK, sV = base + C::kOffV;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kConvW = 8, kProdW = 12, kMmaW = kProdW + 1, kMmaW2 = kProdW + 2;
    volatile int32_t *dead = &ct.dead;
    auto bar = [&](uint64_t &b) { return smem_u32(&b); };
    auto wait = [&](uint64_t &b, uint32_t parity) { return tree_wait(smem_u32(&b), parity, dead, p.err); };

    if (tid == 0) {
        constexpr int kKC = C::kConv ? 4 : 1;                      // who empties a stage: converter warps, or the issuer
        for (int i = 0; i < C::kNK; ++i) mbar_init(bar(ct.kfull[i]), 1), mbar_init(bar(ct.kempty[i]), kKC);
        for (int i = 0; i < C::kNV; ++i) mbar_init(bar(ct.vfull[i]), 1), mbar_init(bar(ct.vempty[i]), kKC);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(ct.k16full[i]), 4), mbar_init(bar(ct.k16empty[i]), 1), mbar_init(bar(ct.v16empty[i]), 1);
            mbar_init(bar(ct.sfull[i]), 1), mbar_init(bar(ct.sempty[i]), 4);
        }
        for (int i = 0; i < C::kNVR; ++i) mbar_init(bar(ct.vready[i]), 4);
        for (int i = 0; i < 2; ++i) mbar_init(bar(ct.pfull[i]), 4), mbar_init(bar(ct.pempty[i]), 1);
        mbar_init(bar(ct.qfull), 4), mbar_init(bar(ct.qempty), 1), mbar_init(bar(ct.oempty), 8), mbar_init(bar(ct.drained[0]), 1), mbar_init(bar(ct.drained[1]), 1);
        for (int i = 0; i < C::kND; ++i)
            mbar_init(bar(ct.dfull[i]), 1), mbar_init(bar(ct.dempty[i]), 8 + 4 + 2), mbar_init(bar(ct.cfull[i]), 4);
        ct.dead = 0;
        fence_mbar_init();
    }
    if (warp == kMmaW) tmem_alloc(smem_u32(&ct.tmem), 512);
    if (C::kConv && kKv == FKV_KV_FP8_E4M3 && warp == kProdW && lane == 0) prefetch_tensormap(&tmK), prefetch_tensormap(&tmV);

    grid_dep_wait();                                               // lengths, tables and cache of earlier kernels
    const int tpt = kR / p.group;                                  // tokens of a unit's rows
    const TreeTotal total = tree_shares<kTreeTok, C::kThreads, 1>(p, tpt, ct.shares);
    const int64_t g0 = total.begin(blockIdx.x), g1 = total.begin(blockIdx.x + 1);
    umma_fence_before();
    __syncthreads();
    umma_fence_after();
    const uint32_t tmem = ct.tmem;
    grid_dep_launch();

    if (warp >= kProdW) {
        if constexpr (C::kShift) regs_down<C::kRegsRest>();
        if (warp == kProdW) {
        // ==== producer ====
        const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_normal();
        int r = ct.shares.r[0];
        int64_t off = ct.shares.off[0], left = g1 - g0;
        int4 join = make_int4(-1, 0, 0, 0);
        TreeRequest cur = tree_request(p, r), nxt = tree_request(p, r + 1);
        Ring d, k, v;
        const int npg = kTreeTok / p.page_size;
        while (left > 0 && !__any_sync(kAll, *dead != 0)) {
            const TreeSpan sp = tree_span<kTreeTok>(p, cur);
            const int mt = (cur.n + tpt - 1) / tpt, units = mt * p.hkv;
            const uint64_t policy = mt > 1 ? again : once;
            for (int ui = static_cast<int>(off / sp.tiles), tb = static_cast<int>(off % sp.tiles); ui < units && left > 0; ++ui, tb = 0) {
                const int te = left < sp.tiles - tb ? tb + static_cast<int>(left) : sp.tiles;
                const int h = ui / mt, m = ui - h * mt;
                wait(ct.dempty[d.i], d.ph ^ 1);
                if (__any_sync(kAll, *dead != 0)) break;           // others may still read what is there
                TreeUnit u;
                u.tb = tb;
                u.te = te;
                u.tok0 = cur.t0 + m * tpt;
                u.ntok = min(tpt, cur.n - m * tpt);
                u.ctx = cur.len - cur.n;
                u.len = cur.len;
                u.start = sp.start;
                u.sink_tiles = sp.sink_tiles;
                u.head = sp.head;
                unit_whole<kTreeTok>(p, u);
                u.row = cur.row;
                u.h = h;
                u.slot = tb == 0 && te == sp.tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (tb == 0 ? 1 : 0);
                u.bad = u.odd = 0;
                if (lane == 0) ct.unit[d.i] = u, ct.qmax[d.i] = 0;
                for (int i = lane; i < 4 * kTreePoison; i += 32) (&ct.poison[d.i][0][0])[i] = 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ct.dfull[d.i]));
                if (tb > 0 && te == sp.tiles) {
                    // the last part of a unit that other CTAs began: its first tile's CTA
                    join = make_int4(static_cast<int>(total.of(g1 - left - tb)), u.tok0, u.ntok, h);
                }
                auto page = [&](int i) -> int32_t {                // this lane's page of tile i; -1: none to copy
                    const uint32_t t = tile_at<kTreeTok>(u, i) + static_cast<uint32_t>(lane) * p.page_size;
                    return lane < npg && t < tile_end(u, i) ? __ldg(p.indices + u.row + t / p.page_size) : -1;
                };
                int32_t pg_next = page(tb);
                for (int i = tb; i < te; ++i) {
                    int32_t pg = pg_next;
                    const bool has = lane < npg && tile_at<kTreeTok>(u, i) + static_cast<uint32_t>(lane) * p.page_size < tile_end(u, i);
                    if (i + 1 < te) pg_next = page(i + 1);
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
                        if (!has) return;
                        if (kKv == FKV_KV_FP4) {
                            const uint32_t sz = p.page_size * kFp4Row;
                            bulk_load_hint(dst + lane * sz, cache + (static_cast<int64_t>(pg) * p.hkv + h) * sz, sz, bar(full), policy);
                        } else {
                            tma_load_4d(dst + lane * p.page_size * 128, tm, bar(full), 0, 0, h, pg, policy);
                            if (kKv == FKV_KV_BF16) tma_load_4d(dst + 16384 + lane * p.page_size * 128, tm, bar(full), 64, 0, h, pg, policy);
                        }
                    };
                    if (__any_sync(kAll, !wait(ct.kempty[k.i], k.ph ^ 1))) break;         // a stage that is still read
                    copy(ct.kfull[k.i], sK + k.i * C::kStageB, &tmK, p.k_cache);
                    k.template next<C::kNK>();
                    if (__any_sync(kAll, !wait(ct.vempty[v.i], v.ph ^ 1))) break;
                    copy(ct.vfull[v.i], sV + v.i * C::kStageB, &tmV, p.v_cache);
                    v.template next<C::kNV>();
                }
                left -= te - tb;
                d.template next<C::kND>();
            }
            off = 0;
            if (left > 0) {
                do {
                    ++r;
                    cur = nxt;
                    nxt = tree_request(p, r + 1);
                } while (r < p.batch && !cur.live);
                if (r >= p.batch) break;
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
        } else if (warp == kMmaW || warp == kMmaW2) {
        // ==== issuers: S = K Q^T, and O += V^T P^T ====
        // A whole warp waits, one lane issues: products and commits come from the same thread.
        constexpr bool kB16 = !C::kConv;
        constexpr uint32_t kHi = umma_desc_hi(1024);
        Ring d;
        if (warp == kMmaW) {
            constexpr uint32_t id = umma_idesc(kB16, false, false, 128, kR);
            const uint32_t lQ = umma_desc_lo(sQ, 16), lK = umma_desc_lo(sK, 16);
            Ring k, sb;
            for (uint32_t units = 0;; ++units) {
                wait(ct.dfull[d.i], d.ph);
                const int tb = *const_cast<volatile int32_t *>(&ct.unit[d.i].tb), te = *const_cast<volatile int32_t *>(&ct.unit[d.i].te);
                if (__any_sync(kAll, te < 0 || *dead != 0)) break;
                if (elect_one()) mbar_arrive(bar(ct.dempty[d.i]));
                d.template next<C::kND>();
                wait(ct.qfull, units & 1);
                for (int i = tb; i < te; ++i) {
                    wait(kB16 ? ct.kfull[k.i] : ct.k16full[k.i], k.ph);
                    wait(ct.sempty[sb.i], sb.ph ^ 1);
                    umma_fence_after();
                    const uint32_t dst = tmem + C::kTmS + sb.i * kR, ta = tmem + k.i * 64, la = lK + k.i * (C::kStageB / 16);
                    __syncwarp();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint64_t b = umma_desc(lQ + (kk >> 2) * (kR * 8) + (kk & 3) * 2, kHi);
                            if (kB16) umma_ss(dst, umma_desc(la + (kk >> 2) * 1024 + (kk & 3) * 2, kHi), b, id, kk > 0);
                            else umma_ts(dst, ta + kk * 8, b, id, kk > 0);
                        }
                        umma_commit(bar(ct.sfull[sb.i]));
                        umma_commit(bar(kB16 ? ct.kempty[k.i] : ct.k16empty[k.i]));
                        if (i + 1 == te) umma_commit(bar(ct.qempty));
                    }
                    __syncwarp();
                    k.template next<kB16 ? C::kNK : 2>();
                    sb.template next<2>();
                }
            }
        } else {
            constexpr uint32_t id = umma_idesc(kB16, kB16, true, 128, kR);
            const uint32_t lP = umma_desc_lo(sP, 16384), lV = umma_desc_lo(sV, 16384);
            Ring v, pb;
            for (uint32_t units = 0;; ++units) {
                wait(ct.dfull[d.i], d.ph);
                const int tb = *const_cast<volatile int32_t *>(&ct.unit[d.i].tb), te = *const_cast<volatile int32_t *>(&ct.unit[d.i].te);
                if (__any_sync(kAll, te < 0 || *dead != 0)) break;
                if (elect_one()) mbar_arrive(bar(ct.dempty[d.i]));
                d.template next<C::kND>();
                if (units) wait(ct.oempty, (units - 1) & 1);
                for (int i = tb; i < te; ++i) {
                    wait(ct.vready[v.i], v.ph);
                    wait(ct.pfull[pb.i], pb.ph);
                    umma_fence_after();
                    const uint32_t lv = lV + v.i * (C::kStageB / 16), lp = lP + pb.i * (C::kPB / 16);
                    const uint32_t dst = tmem + C::kTmO + pb.i * kR;
                    const bool first = i < tb + 2;                        // of a unit and a group: its sums start anew
                    __syncwarp();
                    if (elect_one()) {
#pragma unroll
                        for (int w = 0; w < C::kParts; ++w) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                const uint64_t b = umma_desc(lp + w * (C::kPW / 16) + kk * 128, kHi);
                                const bool add = !first || w > 0 || kk > 0;
                                if (C::kConv) umma_ts(dst, tmem + C::kTmV + v.i * 64 + kk * 8, b, id, add);
                                else umma_ss(dst, umma_desc(lv + kk * 128, kHi), b, id, add);
                            }
                        }
                        umma_commit(bar(ct.pempty[pb.i]));
                        umma_commit(bar(C::kConv ? ct.v16empty[v.i & 1] : ct.vempty[v.i]));
                    }
                    __syncwarp();
                    pb.template next<2>();
                    v.template next<C::kNVR>();
                }
            }
        }
        uint64_t &drained = ct.drained[warp - kMmaW];              // nothing is in flight when the block ends
        __syncwarp();
        if (elect_one()) umma_commit(bar(drained));
        __syncwarp();
        mbar_wait_bounded(bar(drained), 0, kTreeDrainNs);
        }
    } else if (warp >= kConvW) {
        // ==== converters ====
        if constexpr (C::kShift) regs_down<C::kRegsConv>();
        const int ctid = tid & 127, cw = ctid >> 5;
        const uint32_t tlane = static_cast<uint32_t>(32 * cw) << 16;
        Ring d, k, kb, v, vb;
        uint32_t nu = 0;
        while (true) {
            wait(ct.dfull[d.i], d.ph);
            const TreeUnit u = ct.unit[d.i];
            if (group_any(4, u.te < 0 || *dead != 0)) break;       // all four warps or none: they meet at barriers below
            // ---- the unit's Q ----
            wait(ct.qempty, (nu & 1) ^ 1);
            constexpr int kU = kR / 8 < 8 ? kR / 8 : 8;        // rows of a thread at a time
            const int c16 = ctid & 15;
            uint4 x[kU];
            auto load = [&](int r8) {
#pragma unroll
                for (int i = 0; i < kU; ++i) {
                    const int row = (r8 + i) * 8 + (ctid >> 4), tk = row / p.group;
                    x[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (tk < u.ntok)
                        x[i] = __ldg(reinterpret_cast<const uint4 *>(
                                         p.q + (static_cast<int64_t>(u.tok0 + tk) * p.hq + u.h * p.group + (row - tk * p.group)) * 128) + c16);
                }
            };
            float up = 1.f, cs = p.scale_log2;
            if (C::kConv) {
                // by the unit's largest finite element: those down to 2^-32 of it stay exact
                uint32_t big = 0;
#pragma unroll 1
                for (int r8 = 0; r8 < kR / 8; r8 += kU) {
                    load(r8);
#pragma unroll
                    for (int i = 0; i < kU; ++i) {
                        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
                            big = max(big, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                        }
                    }
                }
                big = __reduce_max_sync(kAll, big);
                if (lane == 0) atomicMax(&ct.qmax[d.i], big);
                group_sync(4);
                const QueryPower qp = query_power(*const_cast<volatile uint32_t *>(&ct.qmax[d.i]));
                up = qp.up;
                cs = cs * __ldg(p.k_scale + u.h) * qp.down;
            }
#pragma unroll 1
            for (int r8 = 0; r8 < kR / 8; r8 += kU) {
                if (!C::kConv || kU < kR / 8) load(r8);
#pragma unroll
                for (int i = 0; i < kU; ++i) {
                    const int row = (r8 + i) * 8 + (ctid >> 4);
                    if (C::kConv) {
                        uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = pack_f16x2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xFFFF0000u) * up);
                        x[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    st_shared_v4(sQ + (c16 >> 3) * (kR * 128) + row * 128 + (((c16 & 7) ^ (row & 7)) << 4), x[i]);
                }
            }
            if (ctid == 0) ct.colscale[d.i] = cs;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(ct.qfull));
                mbar_arrive(bar(ct.cfull[d.i]));
            }
            ++nu;
            int odd_tiles = 0;
            for (int i = u.tb; i < u.te; ++i) {
                if (C::kConv) {
                    // ---- K: f16 rows in tensor memory ----
                    wait(ct.kfull[k.i], k.ph);
                    wait(ct.k16empty[kb.i], kb.ph ^ 1);
                    umma_fence_after();
#pragma unroll 1
                    for (int hf = 0; hf < 2; ++hf) {
                        uint32_t f[32];
                        half_row<C::kConv ? kKv : FKV_KV_FP8_E4M3>(sK + k.i * C::kStageB, ctid, hf, f);
                        tmem_store(tmem + tlane + kb.i * 64 + 32 * hf, f);
                    }
                    tmem_store_wait();
                    umma_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(ct.k16full[kb.i]));
                        mbar_arrive(bar(ct.kempty[k.i]));
                    }
                    k.template next<C::kNK>();
                    kb.template next<2>();
                }
                // ---- V: f16 in tensor memory; BF16 as it lies ----
                wait(ct.vfull[v.i], v.ph);
                const uint32_t src = sV + v.i * C::kStageB;
                const bool whole = tile_whole(u, i);
                if (__builtin_expect(!whole, 0)) {
                    if (clean_v<kKv>(src, ctid, tile_at<kTreeTok>(u, i) + ctid < tile_end(u, i))) {
                        atomicOr(&ct.poison[d.i][min(odd_tiles, kTreePoison - 1)][ctid >> 5], 1u << (ctid & 31));
                        *const_cast<volatile int32_t *>(&ct.unit[d.i].odd) = 1;
                    }
                    if (C::kConv) group_sync(5);               // a warp reads tokens of other warps too
                    ++odd_tiles;
                }
                constexpr int kF = C::kConv ? kKv : FKV_KV_FP8_E4M3;
                if (C::kConv) wait(ct.v16empty[vb.i & 1], vb.ph ^ 1);
                if constexpr (C::kConv) {
                    umma_fence_after();
                    convert_v_tmem<kF>(src, tmem + tlane + C::kTmV + vb.i * 64, cw, lane);
                    tmem_store_wait();
                    umma_fence_before();
                }
                if (!whole) fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(ct.vready[vb.i]));
                    if (C::kConv) mbar_arrive(bar(ct.vempty[v.i]));
                }
                v.template next<C::kNV>();
                vb.template next<C::kNVR>();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(ct.dempty[d.i]));
            d.template next<C::kND>();
        }
        // ---- rows of requests without work ----
        __syncwarp();
        for (int r = blockIdx.x; r < p.batch; r += gridDim.x) {
            const TreeRequest q = tree_request(p, r);
            if (!q.rows || q.live) continue;
            uint4 *o = reinterpret_cast<uint4 *>(p.out + static_cast<int64_t>(q.t0) * p.hq * 128);
            const int64_t words = static_cast<int64_t>(q.n) * p.hq * 16;
            for (int64_t i = ctid; i < words; i += 128) o[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    } else {
        // ==== softmax ====
        if constexpr (C::kShift) regs_up<C::kRegsSoft>();
        constexpr int kNC = kR, kLd = kNC < 32 ? kNC : 32;     // columns of a thread, and of a load
        const int g = warp >> 2, wq = warp & 3, tok = tid & 127, barrier = 1 + g;
        const uint32_t tlane = static_cast<uint32_t>(32 * wq) << 16;
        const uint32_t tO = tmem + tlane + C::kTmO;
        const uint32_t sPw = sP + g * C::kPB + tok * 128;
        Ring d;
        uint32_t ph = 0, turn = 0, par = 0;                        // rounds of the group's buffers, whose the next tile is, the unit's parity
        float sum[kNC];
        while (true) {
            wait(ct.dfull[d.i], d.ph);
            if (both_any(*dead != 0)) break;
            const TreeUnit u = ct.unit[d.i];
            if (u.te < 0) break;
            float *const refs = ct.ref[par & 1][g];
            const uint32_t sref = smem_u32(refs);
            if (tok < kNC) refs[tok] = -kTreeNone;
#pragma unroll
            for (int j = 0; j < kNC; ++j) sum[j] = 0.f;
            wait(ct.cfull[d.i], d.ph);
            group_sync(barrier);
            const float cs = *const_cast<volatile float *>(&ct.colscale[d.i]);
            bool had = false;                                      // a tile of this unit
            bool far = false;                                      // a reference so large that products are rounded first
            for (int i = u.tb + static_cast<int>((g ^ turn) & 1); i < u.te; i += 2) {
                const bool whole = tile_whole(u, i);
                uint64_t see = ~0ull;
                if (__builtin_expect(!whole, 0)) see = seen_by<kNC>(p, u, 0, tile_at<kTreeTok>(u, i) + tok, tile_end(u, i));
                wait(ct.sfull[g], ph);
                umma_fence_after();
                const uint32_t ts = tmem + tlane + C::kTmS + g * kR;
                float x[kNC];
                // the columns' logits in log2 units, less their references where kLess; unseen ones -infinity
                auto logits = [&](auto less) {
                    constexpr bool kLess = decltype(less)::value;
#pragma unroll
                    for (int c = 0; c < kNC; c += kLd) tmem_load(ts + c, *reinterpret_cast<float(*)[kLd]>(&x[c]));
                    float cc = cs;
                    if (__builtin_expect(kLess && far, 0)) {
                        asm volatile("" ::: "memory");
#pragma unroll
                        for (int j = 0; j < kNC; ++j) x[j] = __fmul_rn(x[j], cs);
                        cc = 1.f;
                    }
                    const uint64_t cc2 = pack2(cc, cc);
#pragma unroll
                    for (int j = 0; j < kNC; j += 4) {
                        uint64_t a, b;
                        if (kLess) {
                            const float4 r4 = ld_shared_f4(sref + 4 * j);
                            a = fma2(pack2(x[j], x[j + 1]), cc2, pack2(r4.x, r4.y));
                            b = fma2(pack2(x[j + 2], x[j + 3]), cc2, pack2(r4.z, r4.w));
                        } else {
                            a = mul2(pack2(x[j], x[j + 1]), cc2);
                            b = mul2(pack2(x[j + 2], x[j + 3]), cc2);
                        }
                        const float2 e = unpack2(a), f = unpack2(b);
                        x[j] = e.x, x[j + 1] = e.y, x[j + 2] = f.x, x[j + 3] = f.y;
                    }
                    if (__builtin_expect(!whole, 0)) {
                        asm volatile("" ::: "memory");             // a branch: as selects every tile would pay for them
#pragma unroll
                        for (int j = 0; j < kNC; ++j)
                            if (!((see >> j) & 1)) x[j] = -INFINITY;
                    }
                };
                for (int tries = 0;; ++tries) {                    // (again after references have moved)
                    logits(std::true_type{});
                    float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int j = 4; j < kNC; ++j) m4[j & 3] = fmaxf(m4[j & 3], x[j]);
                    const float most = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    if (__builtin_expect(!group_any(barrier, most > kTreeMost<kKv>) || tries == 4, 1)) break;
                    // ---- move the references of the columns that need it ----
                    if (had) wait(ct.pempty[g], ph ^ 1);                      // the sums so far are complete
                    umma_fence_after();
                    float(*const red)[kR] = ct.red[par & 1][g];
                    logits(std::false_type{});
                    spread<kNC, 16>(x, lane, [](float a, float b) { return fmaxf(a, b); });
                    constexpr int kHas = kNC >= 32 ? kNC / 32 : 1, kSame = kNC >= 32 ? 1 : 32 / kNC;
                    if (lane % kSame == 0) {
#pragma unroll
                        for (int j = 0; j < kHas; ++j) red[wq][(lane / kSame) * kHas + j] = x[j];
                    }
                    group_sync(barrier);
                    bool move = false, off = false;
                    if (tok < kNC) {
                        const float z = fmaxf(fmaxf(red[0][tok], red[1][tok]), fmaxf(red[2][tok], red[3][tok])), was = -refs[tok];
                        move = z - was > kTreeMost<kKv>;
                        const float ref = move ? tree_reference<kKv>(z) : was;
                        refs[tok] = -ref;
                        ct.up[g][tok] = move ? ex2(was - ref) : 1.f;
                        off = reference_far(ref);
                    }
                    const bool any = group_any(barrier, move);
                    far = group_any(barrier, off);
                    const uint32_t sup = smem_u32(ct.up[g]);
                    if (any && had) {
#pragma unroll
                        for (int j = 0; j < kNC; j += 4) {
                            const float4 f = ld_shared_f4(sup + 4 * j);
                            sum[j] *= f.x, sum[j + 1] *= f.y, sum[j + 2] *= f.z, sum[j + 3] *= f.w;
                        }
#pragma unroll
                        for (int c = 0; c < kNC; c += 8) {
                            float y[8];
                            uint32_t o[8];
                            tmem_load(tO + g * kR + c, y);
#pragma unroll
                            for (int j = 0; j < 8; j += 4) {
                                const float4 f = ld_shared_f4(sup + 4 * (c + j));
                                o[j] = __float_as_uint(y[j] * f.x), o[j + 1] = __float_as_uint(y[j + 1] * f.y);
                                o[j + 2] = __float_as_uint(y[j + 2] * f.z), o[j + 3] = __float_as_uint(y[j + 3] * f.w);
                            }
                            tmem_store(tO + g * kR + c, o);
                        }
                        tmem_store_wait();
                        umma_fence_before();
                    }
                }
                // ---- weights ----
                umma_fence_before();                               // S is read
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ct.sempty[g]));
                wait(ct.pempty[g], ph ^ 1);
#pragma unroll
                for (int j = 0; j < kNC; j += 8) {
#pragma unroll
                    for (int k = j; k < j + 8; k += 2) {
                        x[k] = ex2(x[k]);
                        x[k + 1] = ex2(x[k + 1]);
                        const float2 t = unpack2(add2(pack2(sum[k], sum[k + 1]), pack2(x[k], x[k + 1])));
                        sum[k] = t.x;
                        sum[k + 1] = t.y;
                    }
                    const uint32_t at = sPw + ((j >> 3) ^ (tok & 7)) * 16;
                    if (C::kConv) {
                        st_shared_v4(at, make_uint4(pack_f16x2(x[j], x[j + 1]), pack_f16x2(x[j + 2], x[j + 3]),
                                                    pack_f16x2(x[j + 4], x[j + 5]), pack_f16x2(x[j + 6], x[j + 7])));
                    } else {
                        // two bf16 words: one alone would round a weight by up to 2^-8
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            // the first word cut off, the second rounded: 2^-17 of a weight are left out
                            const uint32_t e = __float_as_uint(x[j + 2 * b]), f = __float_as_uint(x[j + 2 * b + 1]);
                            hi[b] = prmt(e, f, 0x7632);
                            const float2 r = unpack2(add2(pack2(x[j + 2 * b], x[j + 2 * b + 1]),
                                                          pack2(__uint_as_float((e & 0xFFFF0000u) ^ 0x80000000u), __uint_as_float((f & 0xFFFF0000u) ^ 0x80000000u))));
                            lo[b] = pack_bf16x2(r.x, r.y);
                        }
                        st_shared_v4(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                        st_shared_v4(C::kPW < 128 ? sPw + (((j >> 3) + C::kPW / 16) ^ (tok & 7)) * 16 : at + C::kPW, make_uint4(lo[0], lo[1], lo[2], lo[3]));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ct.pfull[g]));
                had = true;
                ph ^= 1;
            }
            turn += u.te - u.tb;
            // ---- end of this CTA's part of the unit ----
            // sums over the tokens; the groups' sums joined; a group writes half of the columns
            constexpr int kHalf = kR / 2, kPer = kNC >= 32 ? kNC / 32 : 1, kSpan = kNC >= 32 ? 1 : 32 / kNC;
            spread<kNC, 16>(sum, lane, [](float a, float b) { return a + b; });
            if (had) wait(ct.pempty[g], ph ^ 1);                           // all products are done, the weights' buffer is free
            float *const ls = &ct.red[par & 1][g][0][0];
            if (lane % kSpan == 0) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) ls[wq * kNC + (lane / kSpan) * kPer + j] = sum[j];
            }
            both_any(false);
            umma_fence_after();
            const bool wrong = *const_cast<volatile int32_t *>(&ct.unit[d.i].bad) != 0, cut = u.slot >= 0;
            float2 *const part = ct.part + g * kHalf;
            const int c0 = g * kHalf;                              // the columns this group writes
            if (tok < kHalf) {
                float l[2] = {0.f, 0.f}, m[2] = {kTreeNone, kTreeNone};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float *x = &ct.red[par & 1][k][0][0] + c0 + tok;
                    l[k] = (x[0] + x[kNC]) + (x[2 * kNC] + x[3 * kNC]);
                    m[k] = -ct.ref[par & 1][k][c0 + tok];
                }
                const float top = l[0] == 0.f ? m[1] : l[1] == 0.f ? m[0] : fmaxf(m[0], m[1]);
                float f[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) f[k] = l[k] == 0.f ? 0.f : ex2(m[k] - top);
                const float all = f[0] * l[0] + f[1] * l[1];
                if (cut) {
                    if (tok + c0 < u.ntok * p.group)
                        p.part_ml[static_cast<int64_t>(u.slot) * kR + c0 + tok] = make_float2(top, wrong ? -1.f : all);
                } else {
                    const float vs = C::kConv ? __ldg(p.v_scale + u.h) : 1.f;
                    const float n = wrong || all == 0.f ? 0.f : vs / all;
                    f[0] *= n;
                    f[1] *= n;
                }
                part[tok] = make_float2(f[0], f[1]);
            }
            group_sync(barrier);
            const bool both = u.te - u.tb > 1;                     // which groups had tiles
            const bool had0 = both || had == (g == 0), had1 = both || had == (g == 1);
            // the dim of this thread's lane (convert_v_tmem)
            const int dim = 32 * wq + dim_of_lane<kKv>(lane);
            const bool anyodd = *const_cast<volatile int32_t *>(&ct.unit[d.i].odd) != 0;
            int tk = c0 / p.group, hr = c0 - tk * p.group;         // of the column: token and query head
            __nv_bfloat16 *out = p.out + (static_cast<int64_t>(u.tok0 + tk) * p.hq + u.h * p.group + hr) * 128 + dim;
            float *po = p.part_o + (static_cast<int64_t>(cut ? u.slot : 0) * kR + c0) * 128 + dim;
            const int64_t skip = static_cast<int64_t>(p.hq - p.group) * 128;
#pragma unroll 1
            for (int c = 0; c < kHalf && tk < u.ntok; c += 8) {
                float y[8], z[8];
                if (had0) tmem_load(tO + c0 + c, y);
                if (had1) tmem_load(tO + kR + c0 + c, z);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 f = part[c + j];
                    float v = had0 ? y[j] * f.x : 0.f;
                    if (had1) v = fmaf(z[j], f.y, v);
                    y[j] = !cut && f.x == 0.f && f.y == 0.f ? 0.f : v;
                }
                if (__builtin_expect(anyodd && !wrong, 0)) {
                    // NaN and infinities of V that not every row sees: left out of the product, here for those who do
                    int k = 0;
                    for (int i = u.tb; i < u.te; ++i) {
                        const uint32_t t0 = tile_at<kTreeTok>(u, i);
                        if (tile_whole(u, i)) continue;
                        for (int b = 0; b < kTreeTok; ++b) {
                            if (!((*const_cast<volatile uint32_t *>(&ct.poison[d.i][min(k, kTreePoison - 1)][b >> 5]) >> (b & 31)) & 1)) continue;
                            const float add = odd_value<kKv>(p, u, t0 + b, dim);
                            const uint64_t see = seen_by<8>(p, u, c0 + c, t0 + b, tile_end(u, i));
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if ((see >> j) & 1) y[j] += add;
                        }
                        ++k;
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (tk < u.ntok) {
                        if (cut) po[j * 128] = y[j];
                        else *out = __float2bfloat16_rn(y[j]);
                    }
                    out += 128;
                    if (++hr == p.group) {
                        hr = 0;
                        ++tk;
                        out += skip;
                    }
                }
                po += 8 * 128;
            }
            umma_fence_before();
            group_sync(barrier);                                   // references, sums and products are read
            if (lane == 0) {
                mbar_arrive(bar(ct.oempty));
                mbar_arrive(bar(ct.dempty[d.i]));
            }
            ++par;
            d.template next<C::kND>();
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
// joining the parts of a unit that is cut
// ---------------------------------------------------------------------------
// Block (c, y): rows 8y .. of the unit whose last part share c had.  The parts are share c0's
// last one and the first ones of c0 + 1 .. c.  Up to 16 parts: a warp joins a row, 8 loads in
// flight.  A few requests alone are cut into a hundred parts, and a warp that read them
// in turn made their joining the longest part of the call (batch of 4, up to 64k tokens: 30 us,
// 13 now): there each warp first sums parts w, w + 8, ... of four rows.
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(32 * kJoinWarps, 4)
tree_join_kernel(const TreeParams p, int rows) {
    __shared__ __align__(16) float4 part_o[kJoinWarps][4][32];
    __shared__ float part_l[kJoinWarps][4], tops[8];
    __shared__ int wrong[8];
    grid_dep_wait();
    grid_dep_launch();
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 j = p.joins[c];
    const int c0 = j.x, row0 = blockIdx.y * 8, n = min(8, j.z * p.group - row0);
    if (c0 < 0 || n <= 0) return;
    const int parts = c - c0 + 1;
    const float vs = p.v_scale ? __ldg(p.v_scale + j.w) : 1.f;
    auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * c0 + 1 : 2 * (c0 + i)) * rows + row0; };
    auto put = [&](int r, bool none, float l, float4 o) {
        const int row = row0 + r, tk = row / p.group;
        none |= l == 0.f;
        const float g = none ? 0.f : vs / l;
        if (none) o = make_float4(0.f, 0.f, 0.f, 0.f);
        uint2 w;
        w.x = pack_bf16x2(o.x * g, o.y * g);
        w.y = pack_bf16x2(o.z * g, o.w * g);
        reinterpret_cast<uint2 *>(p.out + (static_cast<int64_t>(j.y + tk) * p.hq + j.w * p.group + (row - tk * p.group)) * 128)[lane] = w;
    };
    float top = -INFINITY;
    bool bad = false;
    if (parts <= 2 * kJoinWarps) {
        if (warp >= n) return;
        const float2 ml = lane < parts ? p.part_ml[slot(lane) + warp] : make_float2(0.f, 0.f);
        float4 x[8], o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto load = [&](int b) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (b + k < parts) x[k] = reinterpret_cast<const float4 *>(p.part_o + (slot(b + k) + warp) * 128)[lane];
        };
        load(0);
        if (ml.y != 0.f) top = ml.x;                               // 0: it saw nothing
#pragma unroll
        for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
        bad = __any_sync(kAll, ml.y < 0.f);
        const float f = ml.y == 0.f ? 0.f : ex2(ml.x - top);
        float l = 0.f;
        for (int b = 0;;) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float fk = __shfl_sync(kAll, f, b + k), y = __shfl_sync(kAll, ml.y, b + k);
                if (y == 0.f) continue;
                l = fmaf(fk, y, l);
                o.x = fmaf(fk, x[k].x, o.x), o.y = fmaf(fk, x[k].y, o.y), o.z = fmaf(fk, x[k].z, o.z), o.w = fmaf(fk, x[k].w, o.w);
            }
            if ((b += 8) >= parts) break;
            load(b);
        }
        put(warp, bad, l, o);
        return;
    }
    for (int i = lane; i < parts && warp < n; i += 32) {
        const float2 ml = p.part_ml[slot(i) + warp];
        bad |= ml.y < 0.f;
        if (ml.y != 0.f) top = fmaxf(top, ml.x);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    bad = __any_sync(kAll, bad);
    if (lane == 0) {
        tops[warp] = top;
        wrong[warp] = bad;
    }
#pragma unroll 1
    for (int r0 = 0; r0 < n; r0 += 4) {
        __syncthreads();
        float4 o[4];
        float l = 0.f;                                             // lane r: row r0 + r's
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i = warp; i < parts; i += kJoinWarps) {
            const int64_t at = slot(i) + r0;
            float4 x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r0 + r < n) x[r] = reinterpret_cast<const float4 *>(p.part_o + (at + r) * 128)[lane];
            const float2 ml = lane < 4 && r0 + lane < n ? p.part_ml[at + lane] : make_float2(0.f, 0.f);
            const float f = ml.y == 0.f ? 0.f : ex2(ml.x - tops[r0 + (lane & 3)]);
            l = fmaf(f, ml.y, l);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float fr = __shfl_sync(kAll, f, r);
                if (__shfl_sync(kAll, ml.y, r) == 0.f) continue;
                o[r].x = fmaf(fr, x[r].x, o[r].x), o[r].y = fmaf(fr, x[r].y, o[r].y);
                o[r].z = fmaf(fr, x[r].z, o[r].z), o[r].w = fmaf(fr, x[r].w, o[r].w);
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) part_o[warp][r][lane] = o[r];
        if (lane < 4) part_l[warp][lane] = l;
        __syncthreads();
        if (warp < 4 && r0 + warp < n) {
            float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
            l = 0.f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                const float4 x = part_o[w][warp][lane];
                all.x += x.x, all.y += x.y, all.z += x.z, all.w += x.w;
                l += part_l[w][warp];
            }
            put(r0 + warp, wrong[r0 + warp], l, all);
        }
    }
}

cudaError_t launch_tree_join(const TreeParams &p, int shares, int rows, cudaStream_t st) {
    return launch_pdl(tree_join_kernel, dim3(shares, rows / 8), dim3(32 * kJoinWarps), 0, st, p, rows);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {

constexpr int kMaxDev = 64;
std::mutex g_mu;
unsigned long long g_ready[kMaxDev][3][3];                         // the context in which an instance's shared memory was set

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// A pool as a 4-D tensor; a box is a page's rows of one KV head, `rows` at most (BF16: 64 of their dims).
bool page_map(CUtensorMap *m, const void *pool, bool fp8, int P, int Hkv, int S, int rows) {
    const auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t row = fp8 ? 128 : 256;
    const cuuint64_t dims[4] = {128, static_cast<cuuint64_t>(S), static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(P)};
    const cuuint64_t strides[3] = {row, row * S, row * S * Hkv};
    const cuuint32_t box[4] = {fp8 ? 128u : 64u, static_cast<cuuint32_t>(S < rows ? S : rows), 1u, 1u}, step[4] = {1u, 1u, 1u, 1u};
    return enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(pool), dims, strides, box,
               step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool known_kv(int kv) { return kv == FKV_KV_FP8_E4M3 || kv == FKV_KV_BF16 || kv == FKV_KV_FP4; }

// Rows of a unit: the smallest instance that holds the query heads of the requests' mean
// number of tokens.
// From 128 rows on they lie on M (tree_attn_wide.cu): with 128 that was 126 us instead of 145 over BF16, 117 instead of
// 130 over FP8 and 103 instead of 130 over FP4 when both were measured (16 requests of 8192 tokens, 16 drafted; 113, 112 and
// 104 now); with 64, half of M, 801 instead of 603 (FP8, 64 requests around 16k, 8 drafted).  The mean, not the largest, as
// rows of a unit that are not used cost their products; what a ragged step pays is a second unit for requests above it.
int rows_of(int64_t n_tokens, int64_t batch, int64_t group) {
    const int64_t want = group * ((n_tokens + batch - 1) / (batch > 0 ? batch : 1));
    for (int r = 16; r < 128; r *= 2)
        if (want <= r) return r;
    return want > 128 ? kTreeWideRows : 128;
}

// Which kernel.  Up to 32 rows over FP8 or FP4 the products are little work, and the hand-overs of a tile from warp to warp
// cost more than they save: a window of 4096 over FP8 takes 98 us instead of 115, one of 1024 over 16-token FP4 pages 101
// instead of 176, 64 requests around 16k tokens with up to 4 drafted (32 rows) 457 instead of 486.  Few long requests would
// be served faster by the other kernel, 140 us instead of 145 for 16 of them and 58 instead of 67 for 4 (13 of these are the
// joining of a hundred parts a unit): the rule does not look at the batch.
// BF16 needs no conversions and is read by the tensor cores as it lies.
bool small_call(int kv, int rows) { return kv != FKV_KV_BF16 && rows <= 32; }

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
struct TreeWs {
    size_t joins, ml, o, total;
};
TreeWs tree_ws(int sms, int kv, int rows) {
    const size_t shares = small_call(kv, rows) ? tree_small_shares(sms) : sms;
    TreeWs w;
    w.joins = 0;
    w.ml = align256(sizeof(int4) * shares);
    w.o = align256(w.ml + sizeof(float2) * 2 * shares * rows);
    w.total = align256(w.o + sizeof(float) * 128 * 2 * shares * rows);
    return w;
}

template <int kKv, int kR>
fkv_status launch_tree(const TreeParams &p, int sms, const CUtensorMap &tmK, const CUtensorMap &tmV, cudaStream_t st) {
    constexpr int smem = tree_smem<kKv, kR>();
    static_assert(smem <= 232448, "shared memory of a CTA");
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return FKV_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        constexpr int ri = kR == 16 ? 0 : kR == 32 ? 1 : 2;
        const unsigned long long ctx = current_context_id();
        if (ctx == 0 || g_ready[dev][kKv][ri] != ctx) {
            if (cudaFuncSetAttribute(tree_attn_kernel<kKv, kR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
                return FKV_ERR_CUDA;
            g_ready[dev][kKv][ri] = current_context_id();
        }
    }
    if (launch_pdl(tree_attn_kernel<kKv, kR>, dim3(sms), dim3(TreeCfg<kKv, kR>::kThreads), smem, st, p, tmK, tmV) != cudaSuccess)
        return FKV_ERR_CUDA;
    return launch_tree_join(p, sms, kR, st) == cudaSuccess ? FKV_OK : FKV_ERR_CUDA;
}

template <int kKv>
fkv_status launch_rows(int rows, const TreeParams &p, int sms, const CUtensorMap &tmK, const CUtensorMap &tmV, cudaStream_t st) {
    if constexpr (kKv == FKV_KV_BF16) {                            // few rows of the other types: tree_attn_small.cu
        if (rows == 16) return launch_tree<kKv, 16>(p, sms, tmK, tmV, st);
        if (rows == 32) return launch_tree<kKv, 32>(p, sms, tmK, tmV, st);
    }
    return launch_tree<kKv, 64>(p, sms, tmK, tmV, st);
}

// Both calls.  tree: rows and masks per drafted token; else one token a request.
fkv_status attend(bool tree, const void *q, int32_t n_tokens, int32_t num_q_heads, const void *k_cache, const void *v_cache,
                  int32_t kv_dtype, const float *k_scale, const float *v_scale, int32_t num_pages, int32_t num_kv_heads,
                  int32_t page_size, int32_t head_dim, const int32_t *page_indptr, const int32_t *page_indices, int64_t nnz,
                  const int32_t *seq_lens, int32_t batch, const int32_t *token_indptr, const uint64_t *tree_mask,
                  int32_t mask_words, int32_t window, int32_t sinks, const uint8_t *abort_mask, float sm_scale, void *out,
                  void *workspace, size_t workspace_bytes, void *stream) {
    if (n_tokens < 0 || batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_pages <= 0 || nnz < 0) return FKV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads || window < 0 || sinks < 0 || mask_words < 1) return FKV_ERR_INVALID_ARG;
    if (!known_kv(kv_dtype)) return FKV_ERR_INVALID_ARG;
    if (head_dim != 128 || num_q_heads / num_kv_heads > 128 || mask_words > kTreeMaxWords) return FKV_ERR_UNSUPPORTED;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return FKV_ERR_UNSUPPORTED;
    if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return FKV_ERR_INVALID_ARG;
    if (batch == 0 || n_tokens == 0) return FKV_OK;
    // a page's rows are counted in 32 bits by the 4-bit copies
    if (kv_dtype == FKV_KV_FP4 && static_cast<int64_t>(num_kv_heads) * page_size * FKV_FP4_ROW_BYTES > 0x7FFFFFFF)
        return FKV_ERR_UNSUPPORTED;
    if (!q || !k_cache || !v_cache || !page_indptr || !seq_lens || !out || !workspace) return FKV_ERR_INVALID_ARG;
    if (tree && (!token_indptr || !tree_mask)) return FKV_ERR_INVALID_ARG;
    if (nnz > 0 && !page_indices) return FKV_ERR_INVALID_ARG;
    if (kv_dtype != FKV_KV_BF16 && (!k_scale || !v_scale)) return FKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return FKV_ERR_INVALID_ARG;
    uint32_t *err = device_error_word();
    const int sms = device_sm_count();
    if (!err || sms <= 0) return FKV_ERR_CUDA;
    const int group = num_q_heads / num_kv_heads, rows = rows_of(n_tokens, batch, group);
    const TreeWs w = tree_ws(sms, kv_dtype, rows);
    const bool small = small_call(kv_dtype, rows);
    const int box = small ? kTreeSmallTok : kTreeTok;
    if (workspace_bytes < w.total) return FKV_ERR_INVALID_ARG;
    CUtensorMap tmK = {}, tmV = {};                                // unused by the 4-bit cache's untiled copies
    const bool fp8 = kv_dtype == FKV_KV_FP8_E4M3;
    if (kv_dtype != FKV_KV_FP4 && (!page_map(&tmK, k_cache, fp8, num_pages, num_kv_heads, page_size, box) ||
                                   !page_map(&tmV, v_cache, fp8, num_pages, num_kv_heads, page_size, box)))
        return FKV_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    TreeParams p;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache);
    p.k_scale = kv_dtype == FKV_KV_BF16 ? nullptr : k_scale;
    p.v_scale = kv_dtype == FKV_KV_BF16 ? nullptr : v_scale;
    p.indptr = page_indptr;
    p.indices = page_indices;
    p.seq_lens = seq_lens;
    p.token_indptr = tree ? token_indptr : nullptr;
    p.mask = tree ? tree_mask : nullptr;
    p.abort_mask = abort_mask;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.err = err;
    p.joins = reinterpret_cast<int4 *>(ws + w.joins);
    p.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
    p.part_o = reinterpret_cast<float *>(ws + w.o);
    p.nnz = nnz;
    p.batch = batch;
    p.n_tokens = n_tokens;
    p.hq = num_q_heads;
    p.hkv = num_kv_heads;
    p.group = group;
    p.pages = num_pages;
    p.page_size = page_size;
    p.words = mask_words;
    p.window = window;
    p.sinks = sinks;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (small) return launch_tree_small(p, kv_dtype, rows, sms, tmK, tmV, st);
    if (rows >= 128) return launch_tree_wide(p, kv_dtype, rows, sms, tmK, tmV, st);
    return fp8                         ? launch_rows<FKV_KV_FP8_E4M3>(rows, p, sms, tmK, tmV, st)
           : kv_dtype == FKV_KV_BF16 ? launch_rows<FKV_KV_BF16>(rows, p, sms, tmK, tmV, st)
                                     : launch_rows<FKV_KV_FP4>(rows, p, sms, tmK, tmV, st);
}

}  // namespace
}  // namespace fkv

using namespace fkv;

extern "C" size_t paged_tree_attn_workspace_size(int32_t n_tokens, int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                                 int32_t head_dim, int32_t kv_dtype) {
    if (n_tokens < 0 || batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads) return 0;
    if (head_dim != 128 || !known_kv(kv_dtype) || num_q_heads / num_kv_heads > 128) return 0;
    const int sms = device_sm_count();
    // of any call of up to n_tokens tokens, however many requests they are of: fewer rows can mean more shares
    const int group = num_q_heads / num_kv_heads, most = rows_of(std::max(n_tokens, 1), 1, group);
    size_t need = 0;
    for (int rows = rows_of(1, 1, group); rows <= most && sms > 0; rows *= 2)
        need = std::max(need, tree_ws(sms, kv_dtype, rows).total);
    return need;
}

extern "C" fkv_status paged_tree_attn(const void *q, int32_t n_tokens, int32_t num_q_heads, const void *k_cache,
                                      const void *v_cache, int32_t kv_dtype, const float *k_scale, const float *v_scale,
                                      int32_t num_pages, int32_t num_kv_heads, int32_t page_size, int32_t head_dim,
                                      const int32_t *page_indptr, const int32_t *page_indices, int64_t nnz,
                                      const int32_t *seq_lens, int32_t batch, const int32_t *token_indptr,
                                      const uint64_t *tree_mask, int32_t mask_words, int32_t window, int32_t sinks,
                                      const uint8_t *abort_mask, float sm_scale, void *out, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    return attend(true, q, n_tokens, num_q_heads, k_cache, v_cache, kv_dtype, k_scale, v_scale, num_pages, num_kv_heads, page_size,
                  head_dim, page_indptr, page_indices, nnz, seq_lens, batch, token_indptr, tree_mask, mask_words, window, sinks,
                  abort_mask, sm_scale, out, workspace, workspace_bytes, stream);
}

extern "C" fkv_status paged_window_attn(const void *q, int32_t batch, int32_t num_q_heads, const void *k_cache,
                                        const void *v_cache, int32_t kv_dtype, const float *k_scale, const float *v_scale,
                                        int32_t num_pages, int32_t num_kv_heads, int32_t page_size, int32_t head_dim,
                                        const int32_t *page_indptr, const int32_t *page_indices, int64_t nnz,
                                        const int32_t *seq_lens, int32_t window, int32_t sinks, const uint8_t *abort_mask,
                                        float sm_scale, void *out, void *workspace, size_t workspace_bytes, void *stream) {
    if (window <= 0) return FKV_ERR_INVALID_ARG;
    return attend(false, q, batch, num_q_heads, k_cache, v_cache, kv_dtype, k_scale, v_scale, num_pages, num_kv_heads, page_size,
                  head_dim, page_indptr, page_indices, nnz, seq_lens, batch, nullptr, nullptr, 1, window, sinks, abort_mask, sm_scale,
                  out, workspace, workspace_bytes, stream);
}
