// qcache_attn.cu -- selection attention over the 4-bit KV cache.
//
//   s_t = scale * dot(q[h], K[t]),  o[h] = sum_t p_t V[t] / sum_t p_t,  p_t = exp(s_t - m),
//   weight[slot] = sum over the group's heads and the slot's tokens of p_t / sum p
//
// over the tokens of the distinct selected blocks below n_tokens, with K[t] = ks_t kc_t + km_t and
// V[t] = vs_t vc_t + vm_t (codes 0..15, a scale and a minimum per token and KV head).
//
// Nothing is dequantised.  The products run on the tensor cores over the codes themselves and
// the pairs enter outside of them:
//   s_t  = scale * (ks_t (q . kc_t) + km_t sum(q)),
//   o    = sum_t (p_t vs_t) vc_t + sum_t p_t vm_t.
// A code n in a byte of its own, 0x00..0x0F, is the e4m3 number n 2^-9 (subnormal up to 7, then one
// binade of eight steps), so unpacking 8 codes takes two masks and a shift, and the products with
// them are exact.  The other operands are split into e4m3 terms of 4 significant bits, each
// 2^-4 of the one before, in accumulator columns of their own: two terms hold a bf16 query (8
// bits) exactly, three an fp16 one (11 bits); the weights p_t vs_t of P.V are rounded to the same
// number of terms (to 2^-8 of themselves beside bf16 rows, as a bf16 weight would be; 2^-12
// beside fp16 ones), with steps of 2^-18 (2^-22) of the largest weight at the small end.
//
// One CTA (128 threads) per (query, KV head), four CTAs per SM; tiles of two blocks (128 tokens):
//   1. a thread per token unpacks its K row from shared memory into tensor memory; S = K . Q^T with A
//      from tensor memory (M = 128 tokens, N = 16 heads x terms, K = 128 dims);
//   2. meanwhile a thread per dimension unpacks V^T the same way (the record holds V by dimension);
//   3. a thread per token takes its row of S, p = exp2(y) against a running reference m per head, and
//      writes the weights' terms to shared memory (rows = heads x terms, the swizzled K-major
//      layout of B);
//   4. O += V^T . P^T (M = 128 dims, N = 16 heads x terms, K = 128 tokens).
// The references are lazy.  m[h] and the weights' scale g[h] (a power of two that puts the largest
// p vs seen at 2^4) are taken from the first tile, and change only when a later tile's weight
// would pass 2^8 or its y 30: the barrier before step 4 carries that vote, so an ordinary tile
// has two barriers and no reduction across threads.  Sums of p (in fp32) stay per token
// lane until the end.
//
// Records arrive by bulk copies, one per block, two tiles deep.  What bounds it: see the launcher.
// When units are few, a cluster of 2, 4 or 8 CTAs splits a unit's tiles and combines the partial
// outputs through distributed shared memory.  Every wait is bounded; on expiry the CTA raises
// QSA_FLAG_WAIT_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
#include <cuda.h>

#include <cmath>
#include <mutex>

#include "qcache.cuh"
#include "qsa_device.cuh"
#include "tc_ptx.cuh"

namespace qsa {
namespace {

constexpr int kG = 16;                    // head columns of a unit (heads past the group are zeros)
constexpr int kSel = QSA_ATTN_MAX_K;
constexpr int kThreads = 128;
constexpr int kStages = 2;
constexpr int kStageBytes = 2 * kQRec;
constexpr int kMaxSplit = 8;
constexpr float kTop = 4.0f;              // log2 of the largest weight when the references are set
constexpr float kMostWeight = 256.0f;     // a weight above this moves them (e4m3 holds 448)
constexpr float kMostY = 30.0f;           // and a y above this

constexpr int kTileRows(int terms) { return kG * terms; }   // rows of 128 bytes of an operand B tile

struct QCtrl {
    uint64_t full[kStages];
    uint64_t sbar, obar;
    uint32_t tmem_base;
    int abort;
    int nsel, ntok;
    int32_t sel[kSel];                    // the distinct valid ids, in slot order
    int32_t slot[kSel];                   // and the slots they came from
    alignas(16) float f[kG];              // scale log2(e) 2^9 / (the head's power-of-two scaling of q)
    alignas(16) float qs[kG];             // scale log2(e) sum(q)
    alignas(16) float m[kG];              // reference of the exponents (log2 units)
    alignas(16) float g[kG];              // power of two of the weights
    float top[kG], eg[kG];                // largest log2(p vs) + m seen, log2(g)
    float fl[kG], fo[kG];                 // rescaling of the sums and of the outputs
    uint32_t red[2][4][kG];
    float l[kG], mv[kG];
    float2 ml[kMaxSplit][kG];             // (m, l) of every CTA of a cluster
    float w[kSel][kG];                    // sums of p over a slot's tokens
};

template <int TERMS>
struct QLayout {
    static constexpr int kOffQ = 0;                                   // 1024-byte aligned
    static constexpr int kOffP = kOffQ + kTileRows(TERMS) * 128;
    static constexpr int kOffRing = kOffP + kTileRows(TERMS) * 128;
    static constexpr int kOffCtrl = kOffRing + kStages * kStageBytes;
    static constexpr int kBytes = kOffCtrl + (int)sizeof(QCtrl) + 1024;   // + alignment slack
    // tensor memory: S, O, the unpacked K tile and the unpacked V tile (fp16: one region for both)
    static constexpr uint32_t kN = kG * TERMS;
    static constexpr uint32_t kColO = kN;
    static constexpr uint32_t kColK = TERMS == 2 ? 64 : 96;
    static constexpr uint32_t kColV = 96;
    static constexpr uint32_t kCols = 128;
};
static_assert(QLayout<2>::kOffP % 1024 == 0 && QLayout<3>::kOffP % 1024 == 0, "swizzle atoms");
// four CTAs (and 1 KB each that the system keeps) in an SM's 228 KB
static_assert(4 * (QLayout<3>::kBytes + 1024) <= 228 * 1024, "four CTAs per SM");
// the combine's buffers fit the ring: outputs sent and received, 16 heads x 128 fp32 each
static_assert(2 * kG * kQDim * 4 <= kStages * kStageBytes, "combine buffers");

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
__device__ __forceinline__ float ex2(float x) {   // 2^x, 2 ulp
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two fp32 values to fp16 (b high), fp16 pairs to e4m3 pairs and back (exact).
__device__ __forceinline__ uint32_t to_h2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint16_t h2_to_e4m3(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ uint16_t f2_to_e4m3(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_to_h2(uint16_t e) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(e));
    return r;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t h2_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float h2_lo(uint32_t h) { return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu))); }
__device__ __forceinline__ float h2_hi(uint32_t h) { return __half2float(__ushort_as_half((unsigned short)(h >> 16))); }
constexpr uint32_t kH16 = 0x4C004C00u, kHNeg16 = 0xCC00CC00u;   // (16, 16) and (-16, -16)

// The e4m3 terms of two values: v = t0 + t1 / 16 + t2 / 256, |v| <= 448.
template <int TERMS>
__device__ __forceinline__ void split_terms(float a, float b, uint32_t h, uint16_t (&t)[TERMS]) {
    if constexpr (TERMS == 2) {   // from the fp16 pair h = (a, b): its 11 bits are more than the terms'
        t[0] = h2_to_e4m3(h);
        t[1] = h2_to_e4m3(h2_fma(e4m3_to_h2(t[0]), kHNeg16, h2_mul(h, kH16)));
    } else {                      // the first remainder in fp32; it fits fp16 with bits to spare
        t[0] = f2_to_e4m3(a, b);
        const uint32_t h0 = e4m3_to_h2(t[0]);
        const uint32_t r = to_h2((a - h2_lo(h0)) * 16.0f, (b - h2_hi(h0)) * 16.0f);
        t[1] = h2_to_e4m3(r);
        t[2] = h2_to_e4m3(h2_fma(e4m3_to_h2(t[1]), kHNeg16, h2_mul(r, kH16)));
    }
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *local, int rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    return remote;
}
__device__ __forceinline__ void st_cluster(float4 *local, int rank, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr(local, rank)), "f"(v.x), "f"(v.y),
                 "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void st_cluster(float2 *local, int rank, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(cluster_addr(local, rank)), "f"(v.x), "f"(v.y) : "memory");
}

// Sums of 16 values over the warp's 32 lanes in 16 shuffles: each step halves the values a lane
// holds.  Lanes 2h and 2h + 1 return the sum of value h.
__device__ __forceinline__ float warp_sum16(const float (&x)[kG], int lane) {
    float a[8], b[4], c[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float send = (lane & 16) ? x[i] : x[8 + i], keep = (lane & 16) ? x[8 + i] : x[i];
        a[i] = keep + __shfl_xor_sync(kFull, send, 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float send = (lane & 8) ? a[i] : a[4 + i], keep = (lane & 8) ? a[4 + i] : a[i];
        b[i] = keep + __shfl_xor_sync(kFull, send, 8);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float send = (lane & 4) ? b[i] : b[2 + i], keep = (lane & 4) ? b[2 + i] : b[i];
        c[i] = keep + __shfl_xor_sync(kFull, send, 4);
    }
    const float send = (lane & 2) ? c[0] : c[1], keep = (lane & 2) ? c[1] : c[0];
    const float d = keep + __shfl_xor_sync(kFull, send, 2);
    return d + __shfl_xor_sync(kFull, d, 1);
}

// Every thread waits; the warp is converged behind it (the tcgen05 loads and stores need that).
__device__ __forceinline__ void wait_all(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    mbar_wait(bar, parity, abort_flag);
    __syncwarp();
}

struct QParams {
    QAttnArgs a;
    float scale_log2;
    int split;
};

// F16: rows and queries in fp16 (three terms), otherwise bf16 (two); W: the slots' weights are wanted.
template <bool F16, bool W>
__global__ void __launch_bounds__(kThreads, 4) qattn_kernel(const __grid_constant__ QParams p) {
    constexpr int TERMS = F16 ? 3 : 2;
    using L = QLayout<TERMS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sQ = smem + L::kOffQ, *sP = smem + L::kOffP, *ring = smem + L::kOffRing;
    QCtrl &ct = *reinterpret_cast<QCtrl *>(smem + L::kOffCtrl);
    volatile int *abort_flag = &ct.abort;
    const QAttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = p.split, rank = split > 1 ? (int)cluster_ctarank() : 0;
    const int unit = blockIdx.x / split;
    const int qi = unit / a.n_kv_heads, g = unit - qi * a.n_kv_heads;
    const int group = a.n_heads / a.n_kv_heads, nb_cap = a.capacity / kQBlockTok;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&ct.full[s], 1);
        mbar_init(&ct.sbar, 1);
        mbar_init(&ct.obar, 1);
        ct.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // a programmatic dependent of the work before it: nothing is read, and no tensor memory taken,
    // before that work is complete
    wait_prior_grid();
    __syncwarp();
    if (warp == 0) {
        tmem_alloc(&ct.tmem_base, L::kCols);
        tmem_relinquish();
    } else if (warp == 1) {
        // the query's distinct ids inside its context, in slot order
        const int32_t *ids = a.ids + (size_t)qi * a.k;
        const int32_t r0 = lane < a.k ? ids[lane] : -1;
        const int32_t r1 = lane + 32 < a.k ? ids[lane + 32] : -1;
        int ntok = a.n_tokens[qi];
        if (ntok < 0 || ntok > a.capacity) {
            if (lane == 0 && g == 0 && rank == 0 && a.flags) atomicOr(a.flags, QSA_FLAG_NBLOCKS_CLAMPED);
            ntok = ntok < 0 ? 0 : a.capacity;
        }
        const int nb = (ntok + kQBlockTok - 1) / kQBlockTok;
        const unsigned below = (1u << lane) - 1u;
        const bool in0 = r0 >= 0 && r0 < nb, in1 = r1 >= 0 && r1 < nb;
        const bool bad = (r0 != -1 && !in0) || (r1 != -1 && !in1);
        // every lane takes part in every exchange; the conditions come after it
        const unsigned same0 = __match_any_sync(kFull, r0), same1 = __match_any_sync(kFull, r1);
        bool repeat = false;
        if (a.k > 32)
            for (int i = 0; i < 32; ++i) {
                const int32_t other = __shfl_sync(kFull, r0, i);
                repeat |= other == r1;
            }
        const bool take0 = in0 && (same0 & below) == 0u;
        const bool take1 = in1 && (same1 & below) == 0u && !repeat;
        const unsigned m0 = __ballot_sync(kFull, take0), m1 = __ballot_sync(kFull, take1);
        if (take0) {
            const int at = __popc(m0 & below);
            ct.sel[at] = r0;
            ct.slot[at] = lane;
        }
        if (take1) {
            const int at = __popc(m0) + __popc(m1 & below);
            ct.sel[at] = r1;
            ct.slot[at] = lane + 32;
        }
        if (__any_sync(kFull, bad) && lane == 0 && g == 0 && rank == 0 && a.flags) atomicOr(a.flags, QSA_FLAG_BAD_ID);
        if (lane == 0) {
            ct.nsel = __popc(m0) + __popc(m1);
            ct.ntok = ntok;
        }
        if (W && rank == 0) {   // slots that take no part
            float *w = a.weights + ((size_t)qi * a.n_kv_heads + g) * a.k;
            if (lane < a.k && !take0) w[lane] = 0.0f;
            if (lane + 32 < a.k && !take1) w[lane + 32] = 0.0f;
        }
    }
    {   // the group's queries: eight threads per head, 16 dimensions each
        const int h = tid >> 3, part = tid & 7;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.0f;
        if (h < group) {
            const uint4 *row = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.qa) + qi * a.q_stride +
                                                               (int64_t)(g * group + h) * a.q_head_stride + part * 16);
            const uint4 u[2] = {row[0], row[1]};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[8 * i + 2 * j] = QFmt<F16>::lo(w[j]);
                    x[8 * i + 2 * j + 1] = QFmt<F16>::hi(w[j]);
                }
            }
        }
        uint32_t big = 0u;   // the bits of the largest magnitude (an infinity or a NaN stays the largest)
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            big = max(big, __float_as_uint(x[i]) & 0x7FFFFFFFu);
            sum += x[i];
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            big = max(big, __shfl_xor_sync(kFull, big, o));
            sum += __shfl_xor_sync(kFull, sum, o);
        }
        const bool finite = big < 0x7F800000u;
        // a power of two that puts the largest magnitude into [128, 256)
        const int e = finite && big != 0u ? 7 - ilogbf(__uint_as_float(big)) : 0;
        uint32_t out[TERMS][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v0 = finite ? scalbnf(x[2 * i], e) : 0.0f, v1 = finite ? scalbnf(x[2 * i + 1], e) : 0.0f;
            uint16_t t[TERMS];
            split_terms<TERMS>(v0, v1, to_h2(v0, v1), t);
#pragma unroll
            for (int u = 0; u < TERMS; ++u) {
                if (i & 1) out[u][i >> 1] |= (uint32_t)t[u] << 16;
                else out[u][i >> 1] = t[u];
            }
        }
#pragma unroll
        for (int u = 0; u < TERMS; ++u)
            *reinterpret_cast<uint4 *>(sQ + (u * kG + h) * 128 + ((part ^ (h & 7)) << 4)) =
                make_uint4(out[u][0], out[u][1], out[u][2], out[u][3]);
        if (part == 0) {
            ct.f[h] = finite ? scalbnf(p.scale_log2, 9 - e) : __uint_as_float(0x7FC00000u);
            ct.qs[h] = p.scale_log2 * sum;
            ct.m[h] = 0.0f;
            ct.top[h] = -INFINITY;
        }
    }
    if (W)
        for (int i = tid; i < kSel * kG; i += kThreads) (&ct.w[0][0])[i] = 0.0f;
    fence_proxy_async();   // the queries are read by the tensor core
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ct.tmem_base;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const int nsel = ct.nsel, ntok = ct.ntok;
    // this CTA's tiles: all of them, or a slice of a cluster's split
    const int T = (nsel + 1) >> 1;
    const int p0 = rank * T / split, tl = (rank + 1) * T / split - p0;
    const int b0 = 2 * p0, nloc = min(nsel - b0, 2 * tl);
    const uint8_t *head_cache = static_cast<const uint8_t *>(a.cache) + qrec_offset(g, nb_cap, 0);
    auto fetch = [&](int i) {   // one thread: the records of tile i into its stage
        const int n = min(2, nloc - 2 * i), s = i % kStages;
        mbar_expect_tx(&ct.full[s], (uint32_t)(n * kQRec));
        for (int j = 0; j < n; ++j)
            bulk_load(ring + s * kStageBytes + j * kQRec, head_cache + (size_t)ct.sel[b0 + 2 * i + j] * kQRec, kQRec,
                      &ct.full[s]);
    };
    if (tid == 0)
        for (int i = 0; i < kStages && i < tl; ++i) fetch(i);

    const uint32_t id = idesc(0, 128, L::kN);
    const int half = tid >> 6, tok = tid & 63;
    f32x2 l[kG / 2], mv[kG / 2];
#pragma unroll
    for (int h = 0; h < kG / 2; ++h) l[h] = mv[h] = 0ull;
    float e[kG];

    for (int i = 0; i < tl; ++i) {
        const int s = i % kStages;
        const uint8_t *st = ring + s * kStageBytes;
        if (TERMS == 3 && i > 0) wait_all(&ct.obar, (uint32_t)(i - 1) & 1u, abort_flag);   // V(i - 1) is read
        wait_all(&ct.full[s], (uint32_t)(i / kStages) & 1u, abort_flag);
        // ---- K: this thread's token, 128 codes into 32 columns
        const uint8_t *rec = st + half * kQRec;
        {
            uint32_t lo[16], hi[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint4 x = *reinterpret_cast<const uint4 *>(rec + c * 1024 + tok * 16);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    lo[4 * c + j] = w[j] & 0x0F0F0F0Fu;
                    hi[4 * c + j] = (w[j] >> 4) & 0x0F0F0F0Fu;
                }
            }
            tc_fence_after();
            tmem_st16(tmem + lanes + L::kColK, lo);
            tmem_st16(tmem + lanes + L::kColK + 16, hi);
        }
        const bool vis = 2 * i + half < nloc && ct.sel[b0 + min(2 * i + half, nloc - 1)] * kQBlockTok + tok < ntok;
        const uint32_t kp = vis ? *reinterpret_cast<const uint32_t *>(rec + kQOffKPair + tok * 4) : 0u;
        const uint32_t vp = vis ? *reinterpret_cast<const uint32_t *>(rec + kQOffVPair + tok * 4) : 0u;
        tmem_wait_st();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_f8_ta(tmem, tmem + L::kColK + kk * 8, sdesc(smem_u32(sQ) + kk * 32), id, kk > 0 ? 1u : 0u);
            mma_commit(&ct.sbar);
        }
        __syncwarp();
        // ---- V: this thread's dimension, 128 tokens of the two blocks
        if (TERMS == 2 && i > 0) wait_all(&ct.obar, (uint32_t)(i - 1) & 1u, abort_flag);   // V(i - 1), P(i - 1) are read
        if (TERMS == 3) wait_all(&ct.sbar, (uint32_t)i & 1u, abort_flag);                  // K(i) is read
        {
            uint32_t x[2][16];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(st + b * kQRec + kQOffV + c * 2048 + tid * 16);
                    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[b][4 * c + j] = w[j] & 0x0F0F0F0Fu;
                        x[b][8 + 4 * c + j] = (w[j] >> 4) & 0x0F0F0F0Fu;
                    }
                }
            tc_fence_after();
            tmem_st16(tmem + lanes + L::kColV, x[0]);
            tmem_st16(tmem + lanes + L::kColV + 16, x[1]);
        }
        const float ks = QFmt<F16>::lo(kp), km = QFmt<F16>::hi(kp);
        const float vs = QFmt<F16>::lo(vp), vm = QFmt<F16>::hi(vp);
        const bool all_vis = __all_sync(kFull, vis);
        if (TERMS == 2) wait_all(&ct.sbar, (uint32_t)i & 1u, abort_flag);
        tc_fence_after();
        // y = log2(e) s - m of this token, into e
        auto logits = [&]() {
            uint32_t v[TERMS][16];
#pragma unroll
            for (int u = 0; u < TERMS; ++u) tmem_ld16_nowait(tmem + lanes + u * 16, v[u]);
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < TERMS; ++u) reg_fence(v[u]);
            const f32x2 ks2 = pack2(ks, ks), km2 = pack2(km, km);
#pragma unroll
            for (int h = 0; h < kG / 2; ++h) {
                const float2 m = reinterpret_cast<const float2 *>(ct.m)[h];
                const f32x2 f = reinterpret_cast<const f32x2 *>(ct.f)[h], qs = reinterpret_cast<const f32x2 *>(ct.qs)[h];
                f32x2 t = pack2(__uint_as_float(v[TERMS - 1][2 * h]), __uint_as_float(v[TERMS - 1][2 * h + 1]));
#pragma unroll
                for (int u = TERMS - 2; u >= 0; --u)
                    t = fma2(t, pack2(0.0625f, 0.0625f), pack2(__uint_as_float(v[u][2 * h]), __uint_as_float(v[u][2 * h + 1])));
                t = fma2(mul2(t, f), ks2, fma2(km2, qs, pack2(-m.x, -m.y)));
                unpack2(t, e[2 * h], e[2 * h + 1]);
            }
            if (!all_vis)
#pragma unroll
                for (int h = 0; h < kG; ++h) e[h] = vis ? e[h] : -INFINITY;
        };
        bool renew = i == 0;
        while (true) {
            logits();
            if (renew) {
                // new references: the largest exponent and the largest weight so far, per head
                const float lv = vs == 0.0f ? -INFINITY : lg2(vs);
                uint32_t mine[2] = {0u, 0u};
#pragma unroll
                for (int h = 0; h < kG; ++h) {
                    const uint32_t y = __reduce_max_sync(kFull, score_key(e[h]));
                    const uint32_t r = __reduce_max_sync(kFull, score_key(e[h] + lv));
                    if (lane == h) {
                        mine[0] = y;
                        mine[1] = r;
                    }
                }
                if (lane < kG) {
                    ct.red[0][warp][lane] = mine[0];
                    ct.red[1][warp][lane] = mine[1];
                }
                __syncthreads();
                if (tid < kG) {
                    uint32_t y = 0u, r = 0u;
                    for (int w = 0; w < 4; ++w) {
                        y = max(y, ct.red[0][w][tid]);
                        r = max(r, ct.red[1][w][tid]);
                    }
                    const float m0 = ct.m[tid], rise = key_float(y);
                    const float m1 = i == 0 ? rise : m0 + fmaxf(rise, 0.0f);
                    const float top = fmaxf(ct.top[tid], m0 + key_float(r));
                    // nothing but zero scales so far: any other one will pass the limit
                    const float eg = top == -INFINITY ? 60.0f : fminf(fmaxf(kTop - ceilf(top - m1), -126.0f), 126.0f);
                    const float fl = i == 0 ? 1.0f : exp2f(m0 - m1);
                    ct.fl[tid] = fl;
                    ct.fo[tid] = i == 0 ? 1.0f : fl * exp2f(fminf(fmaxf(eg - ct.eg[tid], -126.0f), 126.0f));
                    ct.m[tid] = m1;
                    ct.top[tid] = top;
                    ct.eg[tid] = eg;
                    ct.g[tid] = exp2f(eg);
                }
                __syncthreads();
                if (i > 0) {   // what is summed so far, to the new references (O(i - 1) is complete)
#pragma unroll
                    for (int h = 0; h < kG / 2; ++h) {
                        const f32x2 fl = reinterpret_cast<const f32x2 *>(ct.fl)[h];
                        l[h] = mul2(l[h], fl);
                        mv[h] = mul2(mv[h], fl);
                    }
                    if (W)
                        for (int j = tid; j < 2 * i * kG; j += kThreads) (&ct.w[0][0])[j] *= ct.fl[j % kG];
                    uint32_t o[16];
#pragma unroll
                    for (int u = 0; u < TERMS; ++u) {
                        tmem_ld16_nowait(tmem + lanes + L::kColO + u * 16, o);
                        tmem_wait_ld();
                        reg_fence(o);
#pragma unroll
                        for (int h = 0; h < kG; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * ct.fo[h]);
                        tmem_st16(tmem + lanes + L::kColO + u * 16, o);
                    }
                }
                logits();
            }
            // p = 2^y, the weights p vs g in terms to shared memory: row head (+ 16 per term), column token
            float most = -INFINITY;
#pragma unroll
            for (int h = 0; h < kG; ++h) most = fmaxf(most, e[h]);
            uint32_t hmax = 0u;
            const f32x2 vs2 = pack2(vs, vs);
#pragma unroll
            for (int h = 0; h < kG / 2; ++h) {
                e[2 * h] = ex2(e[2 * h]);
                e[2 * h + 1] = ex2(e[2 * h + 1]);
                const f32x2 w2 = mul2(mul2(pack2(e[2 * h], e[2 * h + 1]), vs2), reinterpret_cast<const f32x2 *>(ct.g)[h]);
                float w0, w1;
                unpack2(w2, w0, w1);
                const uint32_t h2 = to_h2(w0, w1);
                hmax = h2_max(hmax, h2);
                uint16_t t[TERMS];
                split_terms<TERMS>(w0, w1, h2, t);
                uint8_t *r0 = sP + ((uint32_t)tid ^ (uint32_t)(((2 * h) & 7) << 4)) + (2 * h) * 128;
                uint8_t *r1 = sP + ((uint32_t)tid ^ (uint32_t)(((2 * h + 1) & 7) << 4)) + (2 * h + 1) * 128;
#pragma unroll
                for (int u = 0; u < TERMS; ++u) {
                    r0[u * kG * 128] = (uint8_t)t[u];
                    r1[u * kG * 128] = (uint8_t)(t[u] >> 8);
                }
            }
            const bool over = !renew && (most > kMostY || h2_lo(hmax) > kMostWeight || h2_hi(hmax) > kMostWeight);
            fence_proxy_async();   // the weights are read by the tensor core
            tmem_wait_st();
            tc_fence_before();
            if (!__syncthreads_or(over)) break;
            renew = true;
        }
        if (tid == 0) {
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_f8_ta(tmem + L::kColO, tmem + L::kColV + kk * 8, sdesc(smem_u32(sP) + kk * 32), id,
                          (i | kk) != 0 ? 1u : 0u);
            mma_commit(&ct.obar);
            if (i + kStages < tl) fetch(i + kStages);   // every thread has read this stage
        }
        __syncwarp();
        const f32x2 vm2 = pack2(vm, vm);
#pragma unroll
        for (int h = 0; h < kG / 2; ++h) {
            const f32x2 e2 = pack2(e[2 * h], e[2 * h + 1]);
            l[h] = add2(l[h], e2);
            mv[h] = fma2(e2, vm2, mv[h]);
        }
        if (W) {   // two warps per block: their sum does not depend on which comes first
            const float w = warp_sum16(e, lane);
            if ((lane & 1) == 0 && 2 * i + half < nloc) atomicAdd(&ct.w[2 * i + half][lane >> 1], w);
        }
    }

    // ---- sums over the token lanes
    {
        float x[kG];
#pragma unroll
        for (int h = 0; h < kG / 2; ++h) unpack2(l[h], x[2 * h], x[2 * h + 1]);
        const float ls = warp_sum16(x, lane);
#pragma unroll
        for (int h = 0; h < kG / 2; ++h) unpack2(mv[h], x[2 * h], x[2 * h + 1]);
        const float ms = warp_sum16(x, lane);
        __syncthreads();   // every thread has read ct.red
        if ((lane & 1) == 0) {
            ct.red[0][warp][lane >> 1] = __float_as_uint(ls);
            ct.red[1][warp][lane >> 1] = __float_as_uint(ms);
        }
        __syncthreads();
        if (tid < 2 * kG) {
            const int which = tid >> 4, h = tid & 15;
            float sum = 0.0f;
            for (int w = 0; w < 4; ++w) sum += __uint_as_float(ct.red[which][w][h]);
            (which ? ct.mv : ct.l)[h] = sum;
        }
        __syncthreads();
    }
    const size_t head0 = (size_t)qi * a.n_heads + (size_t)g * group;
    auto put = [&](int h, int d, float x) {
        const size_t at = (head0 + h) * kQDim + d;
        if (a.out_dt == QSA_F32) static_cast<float *>(a.out)[at] = x;
        else static_cast<uint16_t *>(a.out)[at] = (uint16_t)QFmt<F16>::bits(x);
    };
    float *part = reinterpret_cast<float *>(ring);   // split: this CTA's unnormalised output [16][128]
    if (tl > 0) {
        wait_all(&ct.obar, (uint32_t)(tl - 1) & 1u, abort_flag);
        tc_fence_after();
        uint32_t o[TERMS][16];
#pragma unroll
        for (int u = 0; u < TERMS; ++u) tmem_ld16_nowait(tmem + lanes + L::kColO + u * 16, o[u]);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < TERMS; ++u) reg_fence(o[u]);
        // this thread's dimension of every head (a warp's stores for one head are 32 neighbours)
#pragma unroll
        for (int h = 0; h < kG; ++h) {
            float x = __uint_as_float(o[TERMS - 1][h]);
#pragma unroll
            for (int u = TERMS - 2; u >= 0; --u) x = fmaf(x, 0.0625f, __uint_as_float(o[u][h]));
            x = fmaf(x * 512.0f, exp2f(-ct.eg[h]), ct.mv[h]);
            if (split > 1) part[h * kQDim + tid] = x;
            else if (h < group) put(h, tid, x / ct.l[h]);
        }
        tc_fence_before();
    } else if (split == 1) {   // no visible token: o = 0
        for (int h = 0; h < group; ++h) put(h, tid, 0.0f);
    }
    if (tid == 0 && ct.abort) {   // a wait gave up: let what is in flight land before the memory is freed
        for (int i = max(0, tl - kStages); i < tl; ++i) mbar_drain(&ct.full[i % kStages], (uint32_t)(i / kStages) & 1u);
        mbar_drain(&ct.sbar, (uint32_t)(tl - 1) & 1u);
        mbar_drain(&ct.obar, (uint32_t)(tl - 1) & 1u);
        if (a.flags) atomicOr(a.flags, QSA_FLAG_WAIT_TIMEOUT);
    }
    if (split == 1) {
        if (a.lse && tid < group)
            a.lse[head0 + tid] = tl > 0 ? (ct.m[tid] + log2f(ct.l[tid])) * 0.6931471805599453f : -INFINITY;
        if (W && tid < nloc) {
            float w = 0.0f;
            for (int h = 0; h < group; ++h) w += ct.w[tid][h] / ct.l[h];
            a.weights[((size_t)qi * a.n_kv_heads + g) * a.k + ct.slot[tid]] = w;
        }
    }
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, L::kCols);
    }
    if (split > 1) {
        // every CTA sends each head's partial output to the CTA that combines that head, and its (m, l)
        // to all; after the barrier each combines from its own memory
        const int nh = kG / split;
        float *recv = part + kG * kQDim;                             // [split][nh][128]
        const float none = -INFINITY;
        cluster_sync();
        if (tl > 0)
            for (int x = tid; x < kG * 32; x += kThreads) {
                const int h = x >> 5, d4 = x & 31;
                st_cluster(reinterpret_cast<float4 *>(recv + (rank * nh + h % nh) * kQDim) + d4, h / nh,
                           reinterpret_cast<const float4 *>(part)[x]);
            }
        for (int x = tid; x < kG * split; x += kThreads) {
            const int h = x % kG;
            st_cluster(&ct.ml[rank][h], x / kG, make_float2(tl > 0 ? ct.m[h] : none, tl > 0 ? ct.l[h] : 0.0f));
        }
        cluster_sync();
        for (int hh = 0; hh < nh; ++hh) {
            const int h = rank * nh + hh;
            float M = -INFINITY, Lsum = 0.0f, acc = 0.0f;
            for (int r = 0; r < split; ++r)
                if (ct.ml[r][h].y != 0.0f) M = fmaxf(M, ct.ml[r][h].x);
            for (int r = 0; r < split; ++r) {
                const float2 v = ct.ml[r][h];
                if (v.y != 0.0f) {   // a CTA without tiles took no part
                    const float f = exp2f(v.x - M);
                    Lsum = fmaf(f, v.y, Lsum);
                    acc = fmaf(f, recv[(r * nh + hh) * kQDim + tid], acc);
                }
            }
            if (h < group) {
                put(h, tid, Lsum != 0.0f ? acc / Lsum : 0.0f);
                if (a.lse && tid == 0) a.lse[head0 + h] = Lsum != 0.0f ? (M + log2f(Lsum)) * 0.6931471805599453f : -INFINITY;
            }
        }
        if (W) {
            if (tid < kG) {   // this CTA's part of the total, per head
                float M = -INFINITY, Lsum = 0.0f;
                for (int r = 0; r < split; ++r)
                    if (ct.ml[r][tid].y != 0.0f) M = fmaxf(M, ct.ml[r][tid].x);
                for (int r = 0; r < split; ++r)
                    if (ct.ml[r][tid].y != 0.0f) Lsum = fmaf(exp2f(ct.ml[r][tid].x - M), ct.ml[r][tid].y, Lsum);
                ct.fl[tid] = tl > 0 ? exp2f(ct.m[tid] - M) / Lsum : 0.0f;
            }
            __syncthreads();
            if (tid < nloc) {
                float w = 0.0f;
                for (int h = 0; h < group; ++h) w = fmaf(ct.w[tid][h], ct.fl[h], w);
                a.weights[((size_t)qi * a.n_kv_heads + g) * a.k + ct.slot[b0 + tid]] = w;
            }
        }
    }
}

template <bool F16, bool W>
qsa_status launch_as(const QParams &p, int grid, cudaStream_t s) {
    constexpr int kBytes = QLayout<F16 ? 3 : 2>::kBytes;
    static std::mutex mu;
    static bool opted_in[64] = {false};
    int dev = 0;
    qsa_status st = check_cuda(cudaGetDevice(&dev), "cudaGetDevice");
    if (st != QSA_OK) return st;
    if (dev < 0 || dev >= 64) return fail(QSA_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!opted_in[dev]) {
            st = check_cuda(cudaFuncSetAttribute(qattn_kernel<F16, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes),
                            "cudaFuncSetAttribute(4-bit selection attention)");
            if (st != QSA_OK) return st;
            opted_in[dev] = true;
        }
    }
    // always a programmatic dependent: its CTAs wait at entry for the work before them
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, qattn_kernel<F16, W>, p), "qattn_kernel launch");
}

}  // namespace

qsa_status launch_qcache_attention(const QAttnArgs &a, cudaStream_t s) {
    QParams p{};
    p.a = a;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    // few units: split each unit's tiles over a cluster, doubling while the grid stays within two CTAs
    // per SM
    const long long units = (long long)a.nq * a.n_kv_heads;
    const int tiles = (a.k + 1) / 2;
    p.split = 1;
    while (p.split < kMaxSplit && p.split * 2 <= tiles && units * p.split * 2 <= 2ll * num_sms()) p.split *= 2;
    const int grid = (int)(units * p.split);
    if (a.dt == QSA_F16) return a.weights ? launch_as<true, true>(p, grid, s) : launch_as<true, false>(p, grid, s);
    return a.weights ? launch_as<false, true>(p, grid, s) : launch_as<false, false>(p, grid, s);
}

}  // namespace qsa
