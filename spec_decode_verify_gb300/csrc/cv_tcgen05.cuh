// Device wrappers of the tcgen05 instructions (sm_103a): tensor memory, matrix products, and the
// descriptors of operands in shared memory.  Every operand tile here is stored as rows of 64 bf16
// (128 bytes) in the 128-byte swizzle: the 16-byte piece c of row r sits at piece c ^ (r % 8).  A tile
// of more than 64 columns is several such blocks one after the other.  The same bytes serve both
// ways: with the row index as the operand's M or N (K contiguous: "K-major") or as its K (M or N
// contiguous: "MN-major").
#pragma once

#include "cv_device.cuh"

namespace cvk {

__device__ __forceinline__ int swizzled(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }

// Shared-memory operand descriptor: start address (bits 0-13), leading byte offset (16-29) and stride
// byte offset (32-45) in units of 16 bytes, version 1 (46), 128-byte swizzle (61-63: 2).  Only the low word
// depends on the address; a step inside a tile is an addition to it.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // groups of 8 rows 1024 bytes apart
// K-major (the leading offset is not used with a swizzle).
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return ((addr >> 4) & 0x3fff) | (1u << 16); }
// MN-major: blocks of 64 M or N elements `block` bytes apart; the 8-row groups run along K.
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr, uint32_t block) {
    return ((addr >> 4) & 0x3fff) | ((block >> 4) << 16);
}

// Instruction descriptor: bf16 operands, fp32 accumulator, M = 128.
__device__ __forceinline__ constexpr uint32_t mma_desc(int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// One lane of the calling warp, the same every time.  The warp runs the issuing code as a whole, so that its
// addresses and descriptors are uniform; only the instructions below are this lane's alone.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r;
}
// D (tensor memory) = A B (+ D when acc), K = 16 per instruction.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 da, db;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %6, 0;\n"
        " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "r"(kDescHigh), "r"(lead)
        : "memory");
}
// The same with A in tensor memory (two bf16 of a row per 32-bit column).
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 db;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %6, 0;\n mov.b64 db, {%2, %5};\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "r"(kDescHigh), "r"(lead)
        : "memory");
}
// Arrive on `bar` once every tcgen05 operation the lane has issued is complete.
__device__ __forceinline__ void mma_commit(uint32_t lead, uint64_t *bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Tensor memory allocation by one warp; the address lands in shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(addr), "r"(cols) : "memory");
}

#define CV_R4(r, i) "=r"((r)[i]), "=r"((r)[i + 1]), "=r"((r)[i + 2]), "=r"((r)[i + 3])
#define CV_P4(r, i) "+r"((r)[i]), "+r"((r)[i + 1]), "+r"((r)[i + 2]), "+r"((r)[i + 3])
#define CV_P16(r, i) CV_P4(r, i), CV_P4(r, i + 4), CV_P4(r, i + 8), CV_P4(r, i + 12)
#define CV_R16(r, i) CV_R4(r, i), CV_R4(r, i + 4), CV_R4(r, i + 8), CV_R4(r, i + 12)
#define CV_I4(r, i) "r"((r)[i]), "r"((r)[i + 1]), "r"((r)[i + 2]), "r"((r)[i + 3])
#define CV_I16(r, i) CV_I4(r, i), CV_I4(r, i + 4), CV_I4(r, i + 8), CV_I4(r, i + 12)

// 16 columns of the calling warp's 32 lanes; the values are there after tmem_wait_ld on the same array.
__device__ __forceinline__ void tmem_ld16(uint32_t *r, uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n"
        : CV_R16(r, 0)
        : "r"(addr)
        : "memory");
}
// All this thread's loads from tensor memory are complete; the array ties later uses of its values to it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" : CV_P16(r, 0)::"memory");
}
// The same for an array whose loads an earlier tmem_wait_ld has already waited for.
__device__ __forceinline__ void tmem_tie(uint32_t *r) { asm volatile("" : CV_P16(r, 0)::"memory"); }
// 8 columns at each of two addresses, and their wait.
__device__ __forceinline__ void tmem_ld8x2(uint32_t *a, uint32_t *b, uint32_t addr_a, uint32_t addr_b) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n"
        : CV_R4(a, 0), CV_R4(a, 4), CV_R4(b, 0), CV_R4(b, 4)
        : "r"(addr_a), "r"(addr_b)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld8x2(uint32_t *a, uint32_t *b) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" : CV_P4(a, 0), CV_P4(a, 4), CV_P4(b, 0), CV_P4(b, 4)::"memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(addr), CV_I4(r, 0),
                 CV_I4(r, 4)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};\n" ::"r"(addr),
        CV_I16(r, 0)
        : "memory");
}
#undef CV_P4
#undef CV_P16
#undef CV_R4
#undef CV_R16
#undef CV_I4
#undef CV_I16

// Two fp32 values rounded to bf16 in one word, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace cvk
