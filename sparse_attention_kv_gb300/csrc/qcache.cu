// qcache.cu -- writing token rows into the 4-bit KV cache and reading them back.
//
// A row x of 128 values is held as 16 levels between its minimum and its maximum:
//   scale = the least 16-bit value >= (max - min) / 15,
//   code  = (x - min) / scale, rounded half to even,   value = scale * code + min.
// Rounding the scale up keeps code <= 15 and |value - x| <= scale / 2 for every x; the
// minimum is one of the row's values, so it is exact.
//
// One CTA (256 threads) per (KV head, block of 64 tokens), four threads per token: thread
// c of a token holds dimensions 16c .. 16c + 15 and 64 + 16c .. 64 + 16c + 15, which is
// one 16-byte row of K plane c, so K goes from registers to the cache.  V is stored
// dimension-major: its codes pass through shared memory once, and each thread writes
// one 16-byte row of a V plane.  A CTA owns its whole block, so a partial block's other
// tokens (the other nibbles of shared bytes) are merged without atomics.
#include <cfloat>

#include "qcache.cuh"
#include "qsa_device.cuh"

namespace qsa {
namespace {

constexpr int kNT = 256;
constexpr int kPitch = 144;   // bytes per token of the staged V codes (16-byte rows, 4-bank steps)

struct RowPtr {
    const uint8_t *p;
    int64_t token_bytes, head_bytes;
};
struct RowPtrW {
    uint8_t *p;
    int64_t token_bytes, head_bytes;
};

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// (x - lo) / scale rounded half to even, exactly: the difference as an unevaluated sum
// a + e, a first quotient (at most one off), and the sign of the remainder against
// half a step.  Each fp32 step before the last comparison is exact.
__device__ __noinline__ int exact_code(float x, float lo, float scale) {
    const float a = x - lo;
    const float bb = a - x;
    const float e = (x - (a - bb)) + (-lo - bb);
    float c = rintf(__fdiv_rn(a, scale));
    const float r = fmaf(-c, scale, a);
    const float h = 0.5f * scale;
    const bool odd = ((int)c & 1) != 0;
    const float over = (r - h) + e, under = (r + h) + e;
    if (over > 0.0f || (over == 0.0f && odd)) c += 1.0f;
    else if (under < 0.0f || (under == 0.0f && odd)) c -= 1.0f;
    return min(max((int)c, 0), 15);
}

// One thread's 32 values of a row (16 dimensions from 16c, 16 from 64 + 16c).
template <bool F16>
__device__ __forceinline__ void load_row(const uint8_t *row, int c, float (&x)[32]) {
    const uint4 *r = reinterpret_cast<const uint4 *>(row);
    const uint4 a[4] = {r[2 * c], r[2 * c + 1], r[8 + 2 * c], r[8 + 2 * c + 1]};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = QFmt<F16>::lo(w[j]);
            x[8 * i + 2 * j + 1] = QFmt<F16>::hi(w[j]);
        }
    }
}

// The row's codes (one nibble pair per byte: dimension 16c + j low, 64 + 16c + j high)
// and its (scale, minimum) pair; the four threads of a token call it together.
template <bool F16>
__device__ __forceinline__ uint32_t quantise(const float (&x)[32], uint32_t (&packed)[4]) {
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) {
        lo = min_nan(lo, x[i]);
        hi = max_nan(hi, x[i]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(kFull, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(kFull, hi, o));
    }
    // upward at every step: the least 16-bit value >= the exact (max - min) / 15 (15 times a
    // 16-bit value is an fp32 value, so no rounding passes one)
    const float range = __fsub_ru(hi, lo);
    if (!(range <= FLT_MAX)) {   // an infinity, a NaN or too wide: the row reads as NaN
        packed[0] = packed[1] = packed[2] = packed[3] = 0u;
        return F16 ? 0x7E007E00u : 0x7FC07FC0u;
    }
    const uint32_t sbits = QFmt<F16>::bits_up(__fdiv_ru(range, 15.0f));
    const float scale = QFmt<F16>::lo(sbits);
    // the approximate quotient is within 1e-5 of the exact one, so it decides the code
    // unless it lies that near to a half; a subnormal scale has no finite reciprocal
    const bool coarse = scale < 1e-30f;
    const float inv = coarse ? 0.0f : __fdividef(1.0f, scale);
    const float sure = coarse ? -1.0f : 0.4999f;
    uint32_t codes[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float q = (x[i] - lo) * inv;
        const float t = rintf(q);
        codes[i] = (uint32_t)(int)t;
        if (fabsf(q - t) > sure) codes[i] = scale > 0.0f ? (uint32_t)exact_code(x[i], lo, scale) : 0u;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        packed[w] = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            packed[w] |= (codes[4 * w + j] | (codes[16 + 4 * w + j] << 4)) << (8 * j);
    }
    return sbits | (QFmt<F16>::bits(lo) << 16);
}

template <bool F16>
__global__ void __launch_bounds__(kNT) append_kernel(const RowPtr k, const RowPtr v, int n, int first_host,
                                                     const int32_t *first_dev, uint8_t *cache, int nb_cap,
                                                     uint32_t *flags) {
    __shared__ __align__(16) uint8_t tile[kQBlockTok * kPitch];   // V codes, [token][dimension]
    const int tid = threadIdx.x, c = tid & 3, tok = tid >> 2;
    const int g = blockIdx.y;
    const long long first = first_dev ? (long long)*first_dev : (long long)first_host;
    const long long cap = (long long)nb_cap * kQBlockTok;
    if (first_dev && blockIdx.x == 0 && g == 0 && tid == 0 && flags && (first < 0 || first + n > cap))
        atomicOr(flags, QSA_FLAG_NBLOCKS_CLAMPED);
    const long long b64 = (first >= 0 ? first / kQBlockTok : -((kQBlockTok - 1 - first) / kQBlockTok)) + blockIdx.x;
    if (b64 < 0 || b64 >= nb_cap) return;
    const int b = (int)b64;
    const long long i = (long long)b * kQBlockTok + tok - first;   // the row this token takes
    if ((long long)b * kQBlockTok >= first + n) return;
    const bool in = i >= 0 && i < n;
    const bool whole = (long long)b * kQBlockTok >= first && (long long)(b + 1) * kQBlockTok <= first + n;
    uint8_t *rec = cache + qrec_offset(g, nb_cap, b);
    float x[32];
    uint32_t packed[4];
    // rows outside the range are read as zeros: the four threads of a token agree on it
    if (in) {
        load_row<F16>(k.p + i * k.token_bytes + g * k.head_bytes, c, x);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = 0.0f;
    }
    const uint32_t kpair = quantise<F16>(x, packed);
    if (in) {
        *reinterpret_cast<uint4 *>(rec + c * 1024 + tok * 16) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
        if (c == 0) *reinterpret_cast<uint32_t *>(rec + kQOffKPair + tok * 4) = kpair;
        load_row<F16>(v.p + i * v.token_bytes + g * v.head_bytes, c, x);
    }
    const uint32_t vpair = quantise<F16>(x, packed);
    if (in && c == 0) *reinterpret_cast<uint32_t *>(rec + kQOffVPair + tok * 4) = vpair;
    // unpacked to bytes: the low nibbles are dimensions 16c .., the high ones 64 + 16c ..
    uint4 *row = reinterpret_cast<uint4 *>(tile + tok * kPitch);
    row[c] = make_uint4(packed[0] & 0x0F0F0F0Fu, packed[1] & 0x0F0F0F0Fu, packed[2] & 0x0F0F0F0Fu,
                        packed[3] & 0x0F0F0F0Fu);
    row[4 + c] = make_uint4((packed[0] >> 4) & 0x0F0F0F0Fu, (packed[1] >> 4) & 0x0F0F0F0Fu,
                            (packed[2] >> 4) & 0x0F0F0F0Fu, (packed[3] >> 4) & 0x0F0F0F0Fu);
    __syncthreads();
    // V plane p, dimension d: byte j holds token 16p + j (low) and 32 + 16p + j (high)
    const int p = tid >> 7, d = tid & 127;
    uint4 *dst = reinterpret_cast<uint4 *>(rec + kQOffV + p * 2048 + d * 16);
    uint32_t w[4], keep[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        w[q] = keep[q] = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t0 = 16 * p + 4 * q + j;
            w[q] |= (uint32_t)(tile[t0 * kPitch + d] | (tile[(t0 + 32) * kPitch + d] << 4)) << (8 * j);
            const long long i0 = (long long)b * kQBlockTok + t0 - first;
            if (i0 < 0 || i0 >= n) keep[q] |= 0x0Fu << (8 * j);
            if (i0 + 32 < 0 || i0 + 32 >= n) keep[q] |= 0xF0u << (8 * j);
        }
    }
    if (!whole) {
        const uint4 old = *dst;
        const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = (w[q] & ~keep[q]) | (o[q] & keep[q]);
    }
    *dst = make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F16>
__device__ __forceinline__ void store_row(uint8_t *row, int c, const uint32_t (&lo)[4], const uint32_t (&hi)[4],
                                          uint32_t pair) {
    const float scale = QFmt<F16>::lo(pair), mn = QFmt<F16>::hi(pair);
    uint4 *r = reinterpret_cast<uint4 *>(row);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = (half ? hi : lo)[2 * i + (j >> 1)] >> (16 * (j & 1));
                o[j] = QFmt<F16>::bits(fmaf(scale, (float)(w & 0xFFu), mn)) |
                       (QFmt<F16>::bits(fmaf(scale, (float)((w >> 8) & 0xFFu), mn)) << 16);
            }
            r[8 * half + 2 * c + i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
}

template <bool F16>
__global__ void __launch_bounds__(kNT) load_kernel(const uint8_t *cache, int nb_cap, int first, int n,
                                                   const RowPtrW k, const RowPtrW v) {
    __shared__ __align__(16) uint8_t tile[kQBlockTok * kPitch];
    const int tid = threadIdx.x, c = tid & 3, tok = tid >> 2;
    const int g = blockIdx.y, b = first / kQBlockTok + blockIdx.x;
    const uint8_t *rec = cache + qrec_offset(g, nb_cap, b);
    const long long i = (long long)b * kQBlockTok + tok - first;
    const bool in = i >= 0 && i < n;
    uint32_t lo[4], hi[4];
    auto unpack = [&](uint4 x) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            lo[j] = w[j] & 0x0F0F0F0Fu;
            hi[j] = (w[j] >> 4) & 0x0F0F0F0Fu;
        }
    };
    {   // V codes to shared memory, token-major
        const int p = tid >> 7, d = tid & 127;
        unpack(*reinterpret_cast<const uint4 *>(rec + kQOffV + p * 2048 + d * 16));
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            tile[(16 * p + j) * kPitch + d] = (uint8_t)(lo[j >> 2] >> (8 * (j & 3)));
            tile[(32 + 16 * p + j) * kPitch + d] = (uint8_t)(hi[j >> 2] >> (8 * (j & 3)));
        }
    }
    if (in) {
        unpack(*reinterpret_cast<const uint4 *>(rec + c * 1024 + tok * 16));
        store_row<F16>(k.p + i * k.token_bytes + g * k.head_bytes, c, lo, hi,
                       *reinterpret_cast<const uint32_t *>(rec + kQOffKPair + tok * 4));
    }
    __syncthreads();
    if (in) {
        const uint4 a = reinterpret_cast<const uint4 *>(tile + tok * kPitch)[c];
        const uint4 e = reinterpret_cast<const uint4 *>(tile + tok * kPitch)[4 + c];
        lo[0] = a.x, lo[1] = a.y, lo[2] = a.z, lo[3] = a.w;
        hi[0] = e.x, hi[1] = e.y, hi[2] = e.z, hi[3] = e.w;
        store_row<F16>(v.p + i * v.token_bytes + g * v.head_bytes, c, lo, hi,
                       *reinterpret_cast<const uint32_t *>(rec + kQOffVPair + tok * 4));
    }
}

}  // namespace

qsa_status launch_qcache_append(const QAppendArgs &a, cudaStream_t s) {
    const RowPtr k{static_cast<const uint8_t *>(a.k), 2 * a.k_token_stride, 2 * a.k_head_stride};
    const RowPtr v{static_cast<const uint8_t *>(a.v), 2 * a.v_token_stride, 2 * a.v_head_stride};
    // blocks the range touches; from a device position, at most one more than whole ones
    const int blocks = a.first_dev ? (a.n + 2 * kQBlockTok - 2) / kQBlockTok
                                   : (a.first + a.n - 1) / kQBlockTok - a.first / kQBlockTok + 1;
    const dim3 grid((unsigned)blocks, (unsigned)a.n_kv_heads);
    auto *kern = a.dt == QSA_F16 ? append_kernel<true> : append_kernel<false>;
    kern<<<grid, kNT, 0, s>>>(k, v, a.n, a.first, a.first_dev, static_cast<uint8_t *>(a.cache),
                              a.capacity / kQBlockTok, a.flags);
    return check_cuda(cudaGetLastError(), "append_kernel launch");
}

qsa_status launch_qcache_load(const QLoadArgs &a, cudaStream_t s) {
    const RowPtrW k{static_cast<uint8_t *>(a.k), 2 * a.k_token_stride, 2 * a.k_head_stride};
    const RowPtrW v{static_cast<uint8_t *>(a.v), 2 * a.v_token_stride, 2 * a.v_head_stride};
    const int blocks = (a.first + a.n - 1) / kQBlockTok - a.first / kQBlockTok + 1;
    const dim3 grid((unsigned)blocks, (unsigned)a.n_kv_heads);
    auto *kern = a.dt == QSA_F16 ? load_kernel<true> : load_kernel<false>;
    kern<<<grid, kNT, 0, s>>>(static_cast<const uint8_t *>(a.cache), a.capacity / kQBlockTok, a.first, a.n, k, v);
    return check_cuda(cudaGetLastError(), "load_kernel launch");
}

}  // namespace qsa
