// tc_ptx_tmem.cuh -- inline-PTX wrappers beside those of tc_ptx.cuh for kernels that write tensor
// memory from registers: 8-column loads and stores, the 8-bit MMA with A in tensor memory, the
// MN-major operand without swizzle, and the untiled bulk copy.
#pragma once

#include "tc_ptx.cuh"

namespace qsa {

// One contiguous copy; both addresses 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// kind::f8f6f4 with A in tensor memory (`a`: row i of A in lane i, 4 bytes of its K axis per column).
__device__ __forceinline__ void mma_f8_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}
// 8 consecutive columns of this warp's 32 TMEM lanes, one row of 8 values per thread.
__device__ __forceinline__ void tmem_ld8_nowait(uint32_t taddr, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// As tc_ptx.cuh's, for 8 registers.
__device__ __forceinline__ void reg_fence(uint32_t (&v)[8]) {
    asm volatile(""
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]));
}
// Shared-memory matrix descriptor: MN-major operand without swizzle.  16 bytes of the M or N axis
// are contiguous, 8 steps of the K axis lie 16 bytes apart, groups of 8 steps `k_bytes` apart and
// the next 16 bytes of the M or N axis `mn_bytes` apart.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t k_bytes, uint32_t mn_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(k_bytes >> 4) << 16;
    d |= (uint64_t)(mn_bytes >> 4) << 32;
    d |= (uint64_t)1 << 46;
    return d;
}
constexpr uint32_t kIdescBMn = 1u << 16;   // instruction descriptor: B is MN-major

}  // namespace qsa
