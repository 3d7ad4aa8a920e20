// dt_tcgen05.cuh -- fifth-generation tensor core (tcgen05) helpers, sm_100a+.
//
// Tensor memory (TMEM) holds the accumulators: 128 lanes x 512 32-bit columns
// per SM, allocated in power-of-two column blocks by one warp.  An MMA is
// issued by a single thread; its operands are read from shared memory through
// 64-bit matrix descriptors; completion is signalled on an mbarrier with
// tcgen05.commit; the accumulator is read back to registers with tcgen05.ld.
#pragma once

#include "dt_device.cuh"

// ---- TMEM allocation (one full warp) ---------------------------------------
// Allocates ncols columns (power of two, >= 32) and writes the TMEM address to
// the shared-memory word `dst`.
DT_DI void dt_tmem_alloc(uint32_t* dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dt_smem_addr(dst)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
DT_DI void dt_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Ordering of tcgen05 operations around thread synchronisation.
DT_DI void dt_tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
DT_DI void dt_tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Makes this thread's generic-proxy shared-memory writes visible to the async
// proxy (tensor-core operand reads).
DT_DI void dt_fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- shared-memory matrix descriptor -----------------------------------------
// K-major operand tile with 128-byte swizzling: rows of 128 bytes (64 bf16),
// 8-row atoms of 1 KB stacked along M (or N); the tile base is 1024-byte
// aligned.  Row r's 16-byte chunk c is stored at chunk c ^ (r % 8).
// Fields: start address >> 4 (bits 0-13), leading-dimension byte offset >> 4
// (16-29; unused within one 128-byte swizzle span, set to 1), stride byte
// offset >> 4 (32-45: 1024 B between 8-row atoms), descriptor version 1
// (bits 46-47), base offset 0, swizzle mode 2 = 128 B (bits 61-63).
DT_DI uint64_t dt_desc_kmajor_sw128(uint32_t smem_addr) {
    return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Byte offset of element (row r, k) (16-bit elements, k < 64) in such a tile.
DT_DI uint32_t dt_sw128_offset(int r, int k) {
    const uint32_t b = (uint32_t)k * 2u;
    return (uint32_t)r * 128u + ((((b >> 4) ^ (uint32_t)(r & 7)) << 4) | (b & 15u));
}

// ---- instruction descriptor, kind::f16 ---------------------------------------
// bf16 A and B (both K-major), fp32 accumulator, shape M x N:
// D format f32 (bits 4-5 = 1), A format bf16 (7-9 = 1), B format bf16
// (10-12 = 1), no negation, K-major A and B (bits 15, 16 = 0), N >> 3
// (17-22), M >> 4 (24-28).
__host__ __device__ constexpr uint32_t dt_idesc_bf16_f32(int M, int N) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A * B^T for one K step of 16, issued by one thread.
DT_DI void dt_mma_bf16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// Arrives on the mbarrier once every tcgen05 operation issued so far by this
// thread has completed.
DT_DI void dt_mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     dt_smem_addr(bar))
                 : "memory");
}

// 32 consecutive fp32 columns of this thread's TMEM lane (warp w of a
// warpgroup reads lanes 32*(w%4) .. +31; taddr includes that lane offset).
// The load and its completion wait are one asm statement, so no use of the
// registers can be scheduled before the data has arrived.
DT_DI void dt_tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// fp16 products, D[tmem] (+)= A * B for one K step of 16, with A in shared
// memory or in tensor memory (lane = row, two elements per column).  The
// 128-byte-swizzled operands are given by the low words of their descriptors
// (address and leading offset) over a common high word: moving along an operand
// is one 32-bit addition.
#define DT_DESC_HI_SW128 ((1024u >> 4) | (1u << 14) | (2u << 29))
DT_DI uint32_t dt_desc_lo(uint32_t smem_addr, uint32_t lbo) { return (smem_addr >> 4) | ((lbo >> 4) << 16); }
DT_DI void dt_mma_ss_lo(uint32_t tmem_d, uint32_t alo, uint32_t blo, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(tmem_d),
        "r"(alo), "r"(blo), "r"(idesc), "r"((uint32_t)accumulate), "r"(DT_DESC_HI_SW128)
        : "memory");
}
DT_DI void dt_mma_ts_lo(uint32_t tmem_d, uint32_t tmem_a, uint32_t blo, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(tmem_d),
        "r"(tmem_a), "r"(blo), "r"(idesc), "r"((uint32_t)accumulate), "r"(DT_DESC_HI_SW128)
        : "memory");
}

// fp16 A (K-major) and B, fp32 accumulator; B K-major, or MN-major (bit 16).
__host__ __device__ constexpr uint32_t dt_idesc_f16_f32(int M, int N, bool b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// MN-major operand tile with 128-byte swizzling: each K index has rows of 128
// bytes (64 16-bit elements along N), 8 K indices to a 1 KB atom, further K
// atoms 1 KB on (stride byte offset), the next 64 elements of N `lbo` bytes on
// (leading byte offset; 16 for a K-major tile, which does not use it).
// Physically the same layout as the K-major tile of rows of 64 elements.

// 16 fp32 columns of this thread's lane: the load, and the wait that makes the
// registers usable (they pass through it, so nothing reads them earlier).
DT_DI void dt_tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
DT_DI void dt_tmem_ld_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
}
// 16 32-bit columns of this thread's lane to tensor memory.
DT_DI void dt_tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
DT_DI void dt_tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {  // 8 of them
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
DT_DI void dt_tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 64 fp32 columns of this thread's lane, loaded and waited for in one
// statement: the registers come out where the load put them.
DT_DI void dt_tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, "
        "%44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, "
        "%63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
          "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
          "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
          "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr), "r"(taddr + 32)
        : "memory");
}
