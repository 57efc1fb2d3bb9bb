// 5th-generation tensor core (tcgen05) helpers for sm_103a: tensor-memory
// allocation, shared-memory matrix descriptors for the 128-byte-swizzled
// K-major layout, instruction descriptors, MMA issue/commit and TMEM loads
// and stores.  Inline PTX only.
//
// Operand layout used throughout (K-major, 128B swizzle): a tile of R rows x
// 128 bytes (64 bf16 or 32 f32/tf32 values of K per row); row r lives at byte
// r*128 and its 16-byte chunk c is stored at chunk position c ^ (r % 8).
// Tiles start on 1024-byte boundaries; 8-row groups are 1024 bytes apart.
// An operand with more K than one tile holds is a sequence of such tiles.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace gdn {
namespace umma {

// Byte offset of (row, kbyte) inside one swizzled 128-byte-row tile.
__host__ __device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t kbyte) {
    return row * 128u + (kbyte ^ ((row & 7u) << 4));
}

// Shared-memory descriptor: K-major, 128B swizzle, 8-row groups 1024 B apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);          // start address
    d |= (uint64_t)1u << 16;                                 // leading byte offset (unused when swizzled)
    d |= (uint64_t)(1024u >> 4) << 32;                       // stride byte offset
    d |= (uint64_t)1u << 46;                                 // descriptor version for tcgen05
    d |= (uint64_t)2u << 61;                                 // layout: 128-byte swizzle
    return d;
}

// ... and the K-stride of an operand whose rows are not its K: tiles of R rows
// (K) x 64 bf16 (M or N), swizzled as above; 8-row groups 1024 B apart (stride
// byte offset), tiles of the next 64 M or N `tile_bytes` apart (leading byte
// offset).  16 rows of K further: 2048 B.
__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t smem_addr, uint32_t tile_bytes) {
    return (desc_sw128(smem_addr) & ~((uint64_t)0x3FFFu << 16)) | ((uint64_t)(tile_bytes >> 4) << 16);
}

enum : uint32_t { kFmtBF16 = 1u, kFmtTF32 = 2u };

// Added to an instruction descriptor: B's rows are its K (desc_sw128_mn).
constexpr uint32_t kBTransposed = 1u << 16;

// Instruction descriptor: dense, f32 accumulator, both operands K-major.
__host__ __device__ constexpr uint32_t idesc(uint32_t M, uint32_t N, uint32_t fmt) {
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// ---------------------------------------------------------------------------
// tensor memory
// ---------------------------------------------------------------------------
// Warp-collective: allocates ncols columns (power of two >= 32) and writes the
// TMEM base address into *slot (shared memory).
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                 "r"(ncols)
                 : "memory");
}

__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void fence_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void fence_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Issue by a whole warp: one lane is elected inside each block, so the code
// around it stays convergent and operands stay in uniform registers.  (Issued
// under a test of the lane number, each product costs the issuing thread some
// 85 cycles, more than an M = N = 128 product takes.)
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

#define GDN_UMMA_WARP_BEGIN                                                                            \
    "{\n\t.reg .pred w, p, t;\n\t.reg .b64 b;\n\telect.sync _|w, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t" \
    "setp.eq.b32 t, 0, 0;\n\t"

// K = 64 (four instructions) of A and B in one 128-byte-swizzled tile each.
__device__ __forceinline__ void warp_mma_bf16_k64(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(GDN_UMMA_WARP_BEGIN
                 ".reg .b64 a;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
                 "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
                 "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 4;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
                 "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 6;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
                 : "memory");
}

// ... of A in tensor memory (32 columns) and B in one tile.
__device__ __forceinline__ void warp_mma_bf16_tmem_a_k64(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(GDN_UMMA_WARP_BEGIN
                 ".reg .b32 a;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
                 "add.u32 a, %1, 8;\n\tadd.u64 b, %2, 2;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
                 "add.u32 a, %1, 16;\n\tadd.u64 b, %2, 4;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
                 "add.u32 a, %1, 24;\n\tadd.u64 b, %2, 6;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
                 : "memory");
}

// ... of A in one tile and 64 rows (K) of a transposed B.
__device__ __forceinline__ void warp_mma_bf16_k64_bt(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(GDN_UMMA_WARP_BEGIN
                 ".reg .b64 a;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
                 "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 128;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
                 "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 256;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
                 "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 384;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
                 : "memory");
}

// K = 32 of A in tensor memory (16 columns) and a transposed B (rows of K).
__device__ __forceinline__ void warp_mma_bf16_tmem_a_k32(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(GDN_UMMA_WARP_BEGIN
                 ".reg .b32 a;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
                 "add.u32 a, %1, 8;\n\tadd.u64 b, %2, 128;\n\t"
                 "@w tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
                 : "memory");
}

__device__ __forceinline__ void warp_mma_commit(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred w;\n\telect.sync _|w, 0xffffffff;\n\t"
        "@w tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// ---------------------------------------------------------------------------
// MMA issue (one thread) and completion
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
        : "memory");
}

__device__ __forceinline__ void mma_tf32(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
        : "memory");
}

// A operand read from tensor memory (M = 128 lanes, 8 f32 columns per
// instruction, used as tf32); B from shared memory.
__device__ __forceinline__ void mma_tf32_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(id), "r"((uint32_t)acc)
        : "memory");
}

// Arrives once on `bar` when every MMA issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

// ---------------------------------------------------------------------------
// TMEM <-> registers: warp w reaches lanes [32 (w % 4), 32 (w % 4) + 32);
// thread i gets lane 32 (w % 4) + i, 32 consecutive columns from `col`.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t tmem_addr(uint32_t base, uint32_t lane, uint32_t col) {
    return base + (lane << 16) + col;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32]) {
    uint32_t u[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
          "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]),
          "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]),
          "=r"(u[30]), "=r"(u[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(__float_as_uint(r[0])), "r"(__float_as_uint(r[1])), "r"(__float_as_uint(r[2])),
        "r"(__float_as_uint(r[3])), "r"(__float_as_uint(r[4])), "r"(__float_as_uint(r[5])),
        "r"(__float_as_uint(r[6])), "r"(__float_as_uint(r[7])), "r"(__float_as_uint(r[8])),
        "r"(__float_as_uint(r[9])), "r"(__float_as_uint(r[10])), "r"(__float_as_uint(r[11])),
        "r"(__float_as_uint(r[12])), "r"(__float_as_uint(r[13])), "r"(__float_as_uint(r[14])),
        "r"(__float_as_uint(r[15])), "r"(__float_as_uint(r[16])), "r"(__float_as_uint(r[17])),
        "r"(__float_as_uint(r[18])), "r"(__float_as_uint(r[19])), "r"(__float_as_uint(r[20])),
        "r"(__float_as_uint(r[21])), "r"(__float_as_uint(r[22])), "r"(__float_as_uint(r[23])),
        "r"(__float_as_uint(r[24])), "r"(__float_as_uint(r[25])), "r"(__float_as_uint(r[26])),
        "r"(__float_as_uint(r[27])), "r"(__float_as_uint(r[28])), "r"(__float_as_uint(r[29])),
        "r"(__float_as_uint(r[30])), "r"(__float_as_uint(r[31]))
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(__float_as_uint(r[0])), "r"(__float_as_uint(r[1])), "r"(__float_as_uint(r[2])), "r"(__float_as_uint(r[3])),
        "r"(__float_as_uint(r[4])), "r"(__float_as_uint(r[5])), "r"(__float_as_uint(r[6])), "r"(__float_as_uint(r[7])),
        "r"(__float_as_uint(r[8])), "r"(__float_as_uint(r[9])), "r"(__float_as_uint(r[10])),
        "r"(__float_as_uint(r[11])), "r"(__float_as_uint(r[12])), "r"(__float_as_uint(r[13])),
        "r"(__float_as_uint(r[14])), "r"(__float_as_uint(r[15]))
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Round a finite f32 to the nearest tf32 value (10 explicit mantissa bits,
// ties away from zero), returned as f32 bits with the low 13 bits clear: half
// of the dropped bits' weight (bit 12) is added to the magnitude bits, which
// carries into the kept bits exactly when the dropped part is at least half an
// ulp, then the dropped bits are cleared.  Two integer operations at the
// integer pipe's full rate.
__device__ __forceinline__ float to_tf32(float x) {
    return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xFFFFE000u);
}

}  // namespace umma
}  // namespace gdn
