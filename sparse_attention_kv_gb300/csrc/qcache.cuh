// qcache.cuh -- the record of one 64-token block of the 4-bit KV cache (qsa.h,
// "The 4-bit KV cache"), shared by the kernels that write, read and attend over it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "qsa_internal.h"

namespace qsa {

// The record's two halves are each one contiguous copy: [K codes][K pairs][V pairs]
// and [V codes].  Codes lie in planes of 16-byte rows, so that a thread per row reads
// 16 bytes beside its neighbours' (no bank conflict from shared memory, full sectors
// from global memory), and the low nibbles of a row are the 8-bit operand of 16
// consecutive dimensions (K) or tokens (V), the high nibbles that of another 16: a mask
// and a shift unpack a word into two.
constexpr int kQBlockTok = 64;
constexpr int kQDim = 128;
constexpr int kQRec = QSA_QCACHE_BLOCK_BYTES;
constexpr int kQOffKPair = 4096;    // after 4 planes of [64 tokens][16 B]
constexpr int kQOffVPair = 4352;
constexpr int kQOffV = 4608;        // 2 planes of [128 dims][16 B]
static_assert(kQOffV + 4096 == kQRec, "record size");

__host__ __device__ inline size_t qrec_offset(int g, int nb_cap, int b) {
    return ((size_t)g * nb_cap + b) * (size_t)kQRec;
}

// Two fp32 values in one operand.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The 16-bit formats of rows and (scale, minimum) pairs.
template <bool F16>
struct QFmt;
template <>
struct QFmt<false> {
    static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
    static __device__ __forceinline__ uint32_t bits(float x) {
        return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(x));
    }
    // what passes the format's range becomes its largest value; a NaN stays one
    static __device__ __forceinline__ uint32_t bits_sat(float x) {
        uint32_t r;
        asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.bf16.f32 h, %1;\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(r) : "f"(x));
        return r;
    }
    static constexpr uint32_t kMax2 = 0x7F7F7F7Fu;   // a pair of the largest finite value
    static __device__ __forceinline__ uint32_t bits_up(float x) {
        return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_ru(x));
    }
    // of packed pairs; a NaN on either side wins
    static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    // a code n in the low byte of kCodeHigh << 8 is the value kCodeBase + n; kMinusBase2 takes the base away
    static constexpr uint32_t kCodeHigh = 0x43434343u, kOne2 = 0x3F803F80u, kMinusBase2 = 0xC300C300u;   // 128
    static constexpr float kShort = 0x1p-12f;   // see quantise()
};
template <>
struct QFmt<true> {
    static __device__ __forceinline__ float lo(uint32_t w) {
        return __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
    }
    static __device__ __forceinline__ float hi(uint32_t w) {
        return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
    }
    static __device__ __forceinline__ uint32_t bits(float x) { return (uint32_t)__half_as_ushort(__float2half_rn(x)); }
    static __device__ __forceinline__ uint32_t bits_sat(float x) {
        uint32_t r;
        asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.f16.f32 h, %1;\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(r) : "f"(x));
        return r;
    }
    static constexpr uint32_t kMax2 = 0x7BFF7BFFu;
    static __device__ __forceinline__ uint32_t bits_up(float x) {
        return (uint32_t)__half_as_ushort(__float2half_ru(x));
    }
    static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    static constexpr uint32_t kCodeHigh = 0x64646464u, kOne2 = 0x3C003C00u, kMinusBase2 = 0xE400E400u;   // 1024
    static constexpr float kShort = 0x1p-9f;
};

}  // namespace qsa
