// umma.cuh -- thin wrappers of the fifth-generation tensor-core instructions (sm_103a):
// tensor-memory allocation, loads and stores, matrix descriptors, f16/bf16 products with
// fp32 accumulators, and commits to an mbarrier.
#pragma once

#include "fkv_common.cuh"

namespace fkv {

// ---- tensor memory ----
// Addresses: lane in bits 16 .., column in bits 0 ..; a warp reaches the 32 lanes of its
// rank in its group of four.
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
__device__ __forceinline__ void umma_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void umma_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define FKV_R4(r, i) "=f"((r)[i]), "=f"((r)[(i) + 1]), "=f"((r)[(i) + 2]), "=f"((r)[(i) + 3])
#define FKV_R8(r, i) FKV_R4(r, i), FKV_R4(r, (i) + 4)
#define FKV_R16(r, i) FKV_R8(r, i), FKV_R8(r, (i) + 8)
// kN consecutive columns of this thread's lane (complete when the call returns: the wait is
// part of it, so that no use is scheduled before it).
template <int kN>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&r)[kN]) {
    static_assert(kN == 8 || kN == 16 || kN == 32 || kN == 64, "8, 16, 32 or 64 columns");
    if constexpr (kN == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
                     "tcgen05.wait::ld.sync.aligned;" : FKV_R8(r, 0) : "r"(addr) : "memory");
    } else if constexpr (kN == 16) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                     "tcgen05.wait::ld.sync.aligned;" : FKV_R16(r, 0) : "r"(addr) : "memory");
    } else if constexpr (kN == 64) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                     "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
                     "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
                     "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
                     "tcgen05.wait::ld.sync.aligned;" : FKV_R16(r, 0), FKV_R16(r, 16), FKV_R16(r, 32), FKV_R16(r, 48) : "r"(addr) : "memory");
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                     "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
                     "tcgen05.wait::ld.sync.aligned;" : FKV_R16(r, 0), FKV_R16(r, 16) : "r"(addr) : "memory");
    }
}
#undef FKV_R4
#undef FKV_R8
#undef FKV_R16

#define FKV_I4(r, i) "r"((r)[i]), "r"((r)[(i) + 1]), "r"((r)[(i) + 2]), "r"((r)[(i) + 3])
#define FKV_I8(r, i) FKV_I4(r, i), FKV_I4(r, (i) + 4)
#define FKV_I16(r, i) FKV_I8(r, i), FKV_I8(r, (i) + 8)
// 32 or 8 consecutive columns of this thread's lane; tmem_store_wait before they are used.
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 ::"r"(addr), FKV_I16(r, 0), FKV_I16(r, 16) : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), FKV_I8(r, 0) : "memory");
}
// 16 lanes of 32 columns (.16x128b.x8): register 2k is lane l / 4, column 4k + l % 4 of this
// thread l, register 2k + 1 the same of lane 8 + l / 4.
__device__ __forceinline__ void tmem_store_rows(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(addr), FKV_I16(r, 0) : "memory");
}
#undef FKV_I4
#undef FKV_I8
#undef FKV_I16
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- matrix descriptors ----
// A shared-memory operand in the 128-byte swizzle: 16-byte chunk c of 128-byte row r lies at
// chunk c ^ (r % 8).  K-major (a row holds 64 elements of K): `stride` from 8 rows to the
// next 8, `lead` unused.  MN-major (a row holds 64 elements of M or N): `lead` to the next
// 64 of them, `stride` from 8 K rows to the next 8.
// A descriptor's upper word is a constant, its lower one moves with the address by sixteenths
// of bytes: one addition a product, on the issuing thread's critical path.
__host__ __device__ constexpr uint32_t umma_desc_hi(uint32_t stride) { return (stride >> 4) | (1u << 14) | (2u << 29); }
__device__ __forceinline__ uint32_t umma_desc_lo(uint32_t addr, uint32_t lead) { return ((addr >> 4) & 0x3FFFu) | ((lead >> 4) << 16); }
__device__ __forceinline__ uint64_t umma_desc(uint32_t lo, uint32_t hi) { return (static_cast<uint64_t>(hi) << 32) | lo; }
// One lane of the (converged) warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r) :: "memory");
    return r != 0;
}
// Registers of the warps of a group of four: given back to, or taken from, the block's.
template <int kN>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kN)); }
template <int kN>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kN)); }
// f16 (bf16: `bf16`) operands, fp32 accumulators; *_mn: that operand is MN-major.
__host__ __device__ constexpr uint32_t umma_idesc(bool bf16, bool a_mn, bool b_mn, int m, int n) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// D (tensor memory) (+)= A (shared memory) B^T (shared memory), 16 of K; one thread.
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
}
// The same with A in tensor memory (two elements of K a column).
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
}
// An arrival on `bar` when all products this thread has issued are done.
__device__ __forceinline__ void umma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace fkv
