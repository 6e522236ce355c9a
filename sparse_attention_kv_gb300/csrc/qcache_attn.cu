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
constexpr int kH = 8;                     // heads of a thread: two warpgroups share the 16
constexpr int kSel = QSA_ATTN_MAX_K;
constexpr int kThreads = 288;             // two warpgroups and the control warp
constexpr int kWork = 256;
constexpr int kStages = 3;
constexpr int kStageBytes = 2 * kQRec;
constexpr int kMaxSplit = 8;
constexpr float kTop = 4.0f;              // log2 of the largest weight when the references are set
constexpr float kMostWeight = 256.0f;     // a weight above this moves them (e4m3 holds 448)
constexpr float kMostY = 30.0f;           // and a y above this
constexpr float kFaint = 0x1p-60f;        // V scales whose weights never reach kMostWeight before p overflows

struct QCtrl {
    uint64_t full[kStages];
    uint64_t sbar[2], obar;
    uint32_t tmem_base;
    int abort;
    int nsel, ntok;
    int32_t sel[kSel + 1];                // the distinct valid ids, in slot order, then one past every context
    int32_t slot[kSel];                   // and the slots they came from
    alignas(16) float f[kG];              // scale log2(e) 2^9 / (the head's power-of-two scaling of q)
    alignas(16) float qs[kG];             // scale log2(e) sum(q)
    alignas(16) float nm[kG];             // minus the reference of the exponents (log2 units)
    alignas(16) float g[kG];              // power of two of the weights
    alignas(16) float fl[kG];             // rescaling of the sums and of the outputs
    alignas(16) float fo[kG];
    float top[kG], eg[kG];                // largest log2(p vs) + m seen, log2(g)
    float least_g;
    uint32_t red[3][4][kG];
    float sum[3][kG];                     // l, sum of p vm, 16 x what the weights' rounding took away
    float2 ml[kMaxSplit][kG];             // (m, l) of every CTA of a cluster
    float w[kSel][kG];                    // sums of p over a slot's tokens
};

template <int TERMS>
struct QLayout {
    static constexpr int kOffQ = 0;                              // heads x terms rows of 128 bytes, swizzled
    static constexpr int kOffP = kOffQ + kG * TERMS * 128;       // per term [128 tokens][16 heads]
    static constexpr int kTermP = 128 * kG;
    static constexpr int kOffRing = kOffP + TERMS * kTermP;
    static constexpr int kOffCtrl = kOffRing + kStages * kStageBytes;
    static constexpr int kBytes = kOffCtrl + (int)sizeof(QCtrl) + 1024;   // + alignment slack
    // tensor memory: two tiles' S, O (two groups: the leading terms, and the others 16 times as
    // large), the unpacked K tile and the unpacked V tile
    static constexpr uint32_t kColS = 0, kColO = 32, kColK = 64, kColV = 96, kCols = 128;
};
// three CTAs (and 1 KB each that the system keeps) in an SM's 228 KB
static_assert(3 * (QLayout<3>::kBytes + 1024) <= 228 * 1024, "three CTAs per SM");
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
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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

// The e4m3 terms of two weights, at most 448: w = t0 + (t1 + t2) / 16 + what is left.  Two terms: from the
// fp16 pair h = (a, b), whose 11 bits are more than theirs; returns 16 x what is left (exact).
template <int TERMS>
__device__ __forceinline__ uint32_t split_weights(float a, float b, uint32_t h, uint16_t (&t)[TERMS]) {
    if constexpr (TERMS == 2) {
        t[0] = h2_to_e4m3(h);
        const uint32_t r = h2_fma(e4m3_to_h2(t[0]), kHNeg16, h2_mul(h, kH16));
        t[1] = h2_to_e4m3(r);
        return h2_sub(r, e4m3_to_h2(t[1]));
    } else {   // the first remainder in fp32; it fits fp16 with bits to spare
        t[0] = f2_to_e4m3(a, b);
        const uint32_t h0 = e4m3_to_h2(t[0]);
        const uint32_t r = to_h2((a - h2_lo(h0)) * 16.0f, (b - h2_hi(h0)) * 16.0f);
        t[1] = h2_to_e4m3(r);
        t[2] = h2_to_e4m3(h2_sub(r, e4m3_to_h2(t[1])));
        return 0u;
    }
}
// The e4m3 terms of two query values below 256 in an fp16 pair: v = t0 + t1 (+ t2), exact for the format's
// significand down to 2^-10 (bf16) and 2^-7 (fp16) of the head's largest value, to 2^-18 of it below.
template <int TERMS>
__device__ __forceinline__ void split_query(uint32_t h, uint16_t (&t)[TERMS]) {
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
        t[u] = h2_to_e4m3(h);
        h = h2_sub(h, e4m3_to_h2(t[u]));
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

// Sums of 8 values over the warp's 32 lanes in 9 shuffles: the first three steps halve the values
// a lane holds.  Lanes 4h .. 4h + 3 return the sum of value h.
__device__ __forceinline__ float warp_sum8(const float (&x)[kH], int lane) {
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float send = (lane & 16) ? x[i] : x[4 + i], keep = (lane & 16) ? x[4 + i] : x[i];
        a[i] = keep + __shfl_xor_sync(kFull, send, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float send = (lane & 8) ? a[i] : a[2 + i], keep = (lane & 8) ? a[2 + i] : a[i];
        b[i] = keep + __shfl_xor_sync(kFull, send, 8);
    }
    const float send = (lane & 4) ? b[0] : b[1], keep = (lane & 4) ? b[1] : b[0];
    float c = keep + __shfl_xor_sync(kFull, send, 4);
    c += __shfl_xor_sync(kFull, c, 2);
    return c + __shfl_xor_sync(kFull, c, 1);
}

// Every thread waits; the warp is converged behind it (the tcgen05 loads and stores need that).
__device__ __forceinline__ void wait_all(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    mbar_wait(bar, parity, abort_flag);
    __syncwarp();
}

// 2^x for an integer x in [-126, 127].
__device__ __forceinline__ float pow2i(int x) { return __int_as_float((x + 127) << 23); }

// Barriers beside __syncthreads: 1 among the two warpgroups, 2 from the first to the control warp.
__device__ __forceinline__ void work_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void k_ready_arrive() { asm volatile("bar.arrive 2, 160;" ::: "memory"); }
__device__ __forceinline__ void k_ready_wait() { asm volatile("bar.sync 2, 160;" ::: "memory"); }
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

struct QParams {
    QAttnArgs a;
    float scale_log2;
    int split;
};

// F16: rows and queries in fp16 (three terms), otherwise bf16 (two); W: the slots' weights are wanted.
template <bool F16, bool W>
__global__ void __launch_bounds__(kThreads, 3) qattn_kernel(const __grid_constant__ QParams p) {
    constexpr int TERMS = F16 ? 3 : 2;
    using L = QLayout<TERMS>;
    extern __shared__ uint8_t smem_raw[];
    // offset, not rounded as a number: the compiler keeps knowing that this is shared memory
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem + L::kOffQ, *sP = smem + L::kOffP, *ring = smem + L::kOffRing;
    QCtrl &ct = *reinterpret_cast<QCtrl *>(smem + L::kOffCtrl);
    volatile int *abort_flag = &ct.abort;
    const QAttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const int split = p.split, rank = split > 1 ? (int)cluster_ctarank() : 0;
    const int unit = blockIdx.x / split;
    const int qi = unit / a.n_kv_heads, g = unit - qi * a.n_kv_heads;
    const int group = a.n_heads / a.n_kv_heads, nb_cap = a.capacity / kQBlockTok;
    const uint8_t *head_cache = static_cast<const uint8_t *>(a.cache) + qrec_offset(g, nb_cap, 0);
    // one thread: the records of tile i (blocks b0 + 2i, b0 + 2i + 1 of sel) into its stage
    auto fetch = [&](int i, int b0, int nloc) {
        const int n = min(2, nloc - 2 * i), s = i % kStages;
        mbar_expect_tx(&ct.full[s], (uint32_t)(n * kQRec));
        for (int j = 0; j < n; ++j)
            bulk_load(ring + s * kStageBytes + j * kQRec, head_cache + (size_t)ct.sel[b0 + 2 * i + j] * kQRec, kQRec,
                      &ct.full[s]);
    };

    // a programmatic dependent of the work before it: nothing is read, and no tensor memory taken,
    // before that work is complete
    if (warp == 8) {
        if (lane == 0) {
            for (int s = 0; s < kStages; ++s) mbar_init(&ct.full[s], 1);
            mbar_init(&ct.sbar[0], 1);
            mbar_init(&ct.sbar[1], 1);
            mbar_init(&ct.obar, 1);
            ct.abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        wait_prior_grid();
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
        const int nsel = __popc(m0) + __popc(m1);
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
        const bool any_bad = __any_sync(kFull, bad);
        if (lane == 0) {
            ct.sel[nsel] = QSA_MAX_BLOCKS;
            ct.nsel = nsel;
            ct.ntok = ntok;
            if (any_bad && g == 0 && rank == 0 && a.flags) atomicOr(a.flags, QSA_FLAG_BAD_ID);
        }
        __syncwarp();
        if (lane == 0) {   // the first tiles, before anything else is ready
            const int T = (nsel + 1) >> 1, p0 = rank * T / split, tl = (rank + 1) * T / split - p0;
            for (int i = 0; i < kStages && i < tl; ++i) fetch(i, 2 * p0, min(nsel - 2 * p0, 2 * tl));
        }
        __syncwarp();
        tmem_alloc(&ct.tmem_base, L::kCols);
        tmem_relinquish();
        if (W && rank == 0) {   // slots that take no part
            float *w = a.weights + ((size_t)qi * a.n_kv_heads + g) * a.k;
            if (lane < a.k && !take0) w[lane] = 0.0f;
            if (lane + 32 < a.k && !take1) w[lane + 32] = 0.0f;
        }
    } else {   // the group's queries: sixteen threads per head, 8 dimensions each
        if (W)
            for (int i = tid; i < kSel * kG; i += kWork) (&ct.w[0][0])[i] = 0.0f;
        wait_prior_grid();
        const int h = tid >> 4, part = tid & 15;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.0f;
        if (h < group) {
            const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.qa) + qi * a.q_stride +
                                                             (int64_t)(g * group + h) * a.q_head_stride + part * 8);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[2 * j] = QFmt<F16>::lo(w[j]);
                x[2 * j + 1] = QFmt<F16>::hi(w[j]);
            }
        }
        uint32_t big = 0u;   // the bits of the largest magnitude (an infinity or a NaN stays the largest)
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            big = max(big, __float_as_uint(x[i]) & 0x7FFFFFFFu);
            sum += x[i];
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            big = max(big, __shfl_xor_sync(kFull, big, o));
            sum += __shfl_xor_sync(kFull, sum, o);
        }
        const bool finite = big < 0x7F800000u;
        // a power of two that puts the largest magnitude into [128, 256), in two exact steps
        const int e = finite && big != 0u ? 7 - ilogbf(__uint_as_float(big)) : 0;
        const float s0 = pow2i(e >> 1), s1 = pow2i(e - (e >> 1));
        uint32_t out[TERMS][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint16_t t[TERMS];
            split_query<TERMS>(finite ? to_h2(x[2 * i] * s0 * s1, x[2 * i + 1] * s0 * s1) : 0u, t);
#pragma unroll
            for (int u = 0; u < TERMS; ++u) {
                if (i & 1) out[u][i >> 1] |= (uint32_t)t[u] << 16;
                else out[u][i >> 1] = t[u];
            }
        }
#pragma unroll
        for (int u = 0; u < TERMS; ++u)
            *reinterpret_cast<uint2 *>(sQ + (u * kG + h) * 128 + (((part >> 1) ^ (h & 7)) << 4) + (part & 1) * 8) =
                make_uint2(out[u][0], out[u][1]);
        if (part == 0) {
            ct.f[h] = finite ? scalbnf(p.scale_log2, 9 - e) : __uint_as_float(0x7FC00000u);
            ct.qs[h] = p.scale_log2 * sum;
            ct.nm[h] = 0.0f;
            ct.top[h] = -INFINITY;
        }
    }
    fence_proxy_async();   // the queries are read by the tensor core
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ct.tmem_base;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int nsel = ct.nsel, ntok = ct.ntok;
    // this CTA's tiles: all of them, or a slice of a cluster's split
    const int T = (nsel + 1) >> 1;
    const int p0 = rank * T / split, tl = (rank + 1) * T / split - p0;
    const int b0 = 2 * p0, nloc = min(nsel - b0, 2 * tl);
    // Two warpgroups: both hold every token of a tile (and every dimension of O), one head half each.
    // The first unpacks K, the second V.
    const int wg = tid >> 7, row = tid & 127, half = row >> 6, tok = row & 63;
    const int h0 = wg * kH;
    f32x2 l[kH / 2], mv[kH / 2];
    uint32_t left[kH / 2];                // fp16 pairs: 16 x what the rounding of this token's weights left
#pragma unroll
    for (int h = 0; h < kH / 2; ++h) {
        l[h] = mv[h] = 0ull;
        left[h] = 0u;
    }
    float e[kH];

    if (warp == 8) {
        // ---- control: S(i + 1) as soon as K(i + 1) is unpacked, O += P(i) V(i) when P(i) stands
        const uint32_t id16 = idesc(0, 128, kG);
        const uint64_t dq = sdesc(smem_u32(sQ)), dp = sdesc_mn(smem_u32(sP), 8 * kG, L::kTermP);
        auto scores = [&](int i) {
            k_ready_wait();
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int u = 0; u < TERMS; ++u)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)   // descriptors count in units of 16 bytes
                        mma_f8_ta(tmem + L::kColS + (i & 1) * kG, tmem + L::kColK + kk * 8, dq + u * (kG * 8) + kk * 2, id16,
                                  (u | kk) != 0 ? 1u : 0u);
                mma_commit(&ct.sbar[i & 1]);
            }
            __syncwarp();
        };
        if (tl > 0) scores(0);
        for (int i = 0; i < tl; ++i) {
            if (i + 1 < tl) scores(i + 1);
            while (__syncthreads_or(0)) {}   // again while the references move
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)   // both groups of columns
                    mma_f8_ta(tmem + L::kColO, tmem + L::kColV + kk * 8, dp + kk * (2 * kG), idesc(0, 128, 2 * kG) | kIdescBMn,
                              (i | kk) != 0 ? 1u : 0u);
                if (TERMS == 3)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8_ta(tmem + L::kColO + kG, tmem + L::kColV + kk * 8, dp + 2 * (L::kTermP / 16) + kk * (2 * kG),
                                  id16 | kIdescBMn, 1u);
                mma_commit(&ct.obar);
                if (i + kStages < tl) fetch(i + kStages, b0, nloc);   // every thread has read this stage
            }
            __syncwarp();
        }
    } else {
    auto wait_full = [&](int i) { wait_all(&ct.full[i % kStages], (uint32_t)(i / kStages) & 1u, abort_flag); };
    // 16 bytes of codes to 4 + 4 columns of a row of A
    uint32_t lo[8], hi[8];
    auto unpack = [&](const uint8_t *src, int at) {
        const uint4 x = *reinterpret_cast<const uint4 *>(src);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            lo[at + j] = w[j] & 0x0F0F0F0Fu;
            hi[at + j] = (w[j] >> 4) & 0x0F0F0F0Fu;
        }
    };
    auto unpack_k = [&](int i) {              // this thread's token, its 128 dimensions
        wait_full(i);
        tc_fence_after();
        const uint8_t *src = ring + (i % kStages) * kStageBytes + half * kQRec + tok * 16;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            unpack(src + (2 * c) * 1024, 0);
            unpack(src + (2 * c + 1) * 1024, 4);
            tmem_st8(tmem + lanes + L::kColK + c * 8, lo);
            tmem_st8(tmem + lanes + L::kColK + 16 + c * 8, hi);
        }
        tmem_wait_st();
        tc_fence_before();
        k_ready_arrive();
    };
    if (wg == 0 && tl > 0) unpack_k(0);
    for (int i = 0; i < tl; ++i) {
        const uint8_t *st = ring + (i % kStages) * kStageBytes;
        const uint8_t *rec = st + half * kQRec;
        if (wg == 0) {
            wait_all(&ct.sbar[i & 1], (uint32_t)(i >> 1) & 1u, abort_flag);   // S(i) is complete, K(i) read
            if (i + 1 < tl) unpack_k(i + 1);
            if (i > 0) wait_all(&ct.obar, (uint32_t)(i - 1) & 1u, abort_flag);   // P(i - 1) is read
        } else {
            wait_full(i);
            if (i > 0) wait_all(&ct.obar, (uint32_t)(i - 1) & 1u, abort_flag);   // V(i - 1), P(i - 1) are read
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {     // this thread's dimension, the tokens of the two blocks
                const uint8_t *src = st + b * kQRec + kQOffV + row * 16;
                unpack(src, 0);
                unpack(src + 2048, 4);
                tmem_st8(tmem + lanes + L::kColV + b * 16, lo);
                tmem_st8(tmem + lanes + L::kColV + b * 16 + 8, hi);
            }
            wait_all(&ct.sbar[i & 1], (uint32_t)(i >> 1) & 1u, abort_flag);
        }
        tc_fence_after();
        const bool vis = ct.sel[b0 + 2 * i + half] * kQBlockTok + tok < ntok;
        const uint32_t kp = vis ? *reinterpret_cast<const uint32_t *>(rec + kQOffKPair + tok * 4) : 0u;
        const uint32_t vp = vis ? *reinterpret_cast<const uint32_t *>(rec + kQOffVPair + tok * 4) : 0u;
        const float ks = QFmt<F16>::lo(kp), km = QFmt<F16>::hi(kp);
        const float vs = QFmt<F16>::lo(vp), vm = QFmt<F16>::hi(vp);
        const bool all_vis = __all_sync(kFull, vis);
        // y = log2(e) s - m of this token, into e
        auto logits = [&]() {
            uint32_t v[kH];
            tmem_ld8_nowait(tmem + lanes + L::kColS + (i & 1) * kG + h0, v);
            tmem_wait_ld();
            reg_fence(v);
            const f32x2 ks2 = pack2(ks, ks), km2 = pack2(km, km);
#pragma unroll
            for (int h = 0; h < kH / 2; h += 2) {
                const ulonglong2 nm = *reinterpret_cast<const ulonglong2 *>(ct.nm + h0 + 2 * h);
                const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(ct.f + h0 + 2 * h);
                const ulonglong2 qs = *reinterpret_cast<const ulonglong2 *>(ct.qs + h0 + 2 * h);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int x = 2 * (h + j);
                    f32x2 t = pack2(__uint_as_float(v[x]), __uint_as_float(v[x + 1]));
                    t = fma2(mul2(t, j ? f.y : f.x), ks2, fma2(km2, j ? qs.y : qs.x, j ? nm.y : nm.x));
                    unpack2(t, e[x], e[x + 1]);
                }
            }
            if (!all_vis)
#pragma unroll
                for (int h = 0; h < kH; ++h) e[h] = vis ? e[h] : -INFINITY;
        };
        bool renew = i == 0;
        while (true) {
            logits();
            if (renew) {
                // new references: the largest exponent and the largest weight so far, per head
                const float lv = vs == 0.0f ? -INFINITY : lg2(vs);
                uint32_t mine[2] = {0u, 0u};
#pragma unroll
                for (int h = 0; h < kH; ++h) {
                    const uint32_t y = __reduce_max_sync(kFull, score_key(e[h]));
                    const uint32_t r = __reduce_max_sync(kFull, score_key(e[h] + lv));
                    if (lane == h) {
                        mine[0] = y;
                        mine[1] = r;
                    }
                }
                if (lane < kH) {
                    ct.red[0][warp & 3][h0 + lane] = mine[0];
                    ct.red[1][warp & 3][h0 + lane] = mine[1];
                }
                work_barrier();
                if (warp == 0) {
                    const int h = lane & 15;
                    uint32_t y = 0u, r = 0u;
                    for (int w = 0; w < 4; ++w) {
                        y = max(y, ct.red[0][w][h]);
                        r = max(r, ct.red[1][w][h]);
                    }
                    const float m0 = -ct.nm[h], rise = key_float(y);
                    const float m1 = i == 0 ? rise : m0 + fmaxf(rise, 0.0f);
                    const float top = fmaxf(ct.top[h], m0 + key_float(r));
                    // nothing but zero scales so far: any other one will pass the limit
                    const float eg = top == -INFINITY ? 60.0f : fminf(fmaxf(kTop - ceilf(top - m1), -126.0f), 126.0f);
                    const float fl = i == 0 ? 1.0f : exp2f(m0 - m1);
                    const float fo = i == 0 ? 1.0f : fl * exp2f(fminf(fmaxf(eg - ct.eg[h], -126.0f), 126.0f));
                    float least = eg;
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(kFull, least, o));
                    __syncwarp();
                    if (lane < kG) {
                        ct.fl[h] = fl;
                        ct.fo[h] = fo;
                        ct.nm[h] = -m1;
                        ct.top[h] = top;
                        ct.eg[h] = eg;
                        ct.g[h] = exp2f(eg);
                        if (lane == 0) ct.least_g = exp2f(least);
                    }
                }
                work_barrier();
                if (i > 0) {   // what is summed so far, to the new references (O(i - 1) is complete)
#pragma unroll
                    for (int h = 0; h < kH / 2; ++h) {
                        const f32x2 fl = reinterpret_cast<const f32x2 *>(ct.fl + h0)[h];
                        const float2 fo = reinterpret_cast<const float2 *>(ct.fo + h0)[h];
                        l[h] = mul2(l[h], fl);
                        mv[h] = mul2(mv[h], fl);
                        if (TERMS == 2) left[h] = to_h2(h2_lo(left[h]) * fo.x, h2_hi(left[h]) * fo.y);
                    }
                    if (W)
                        for (int j = tid; j < 2 * i * kG; j += kWork) (&ct.w[0][0])[j] *= ct.fl[j % kG];
                    uint32_t o[kH];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        tmem_ld8_nowait(tmem + lanes + L::kColO + u * kG + h0, o);
                        tmem_wait_ld();
                        reg_fence(o);
#pragma unroll
                        for (int h = 0; h < kH; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * ct.fo[h0 + h]);
                        tmem_st8(tmem + lanes + L::kColO + u * kG + h0, o);
                    }
                }
                logits();
            }
            // p = 2^y, and the weights p vs g in terms to shared memory: [term][token][head]
            bool over = false;
            if (__any_sync(kFull, vis && vs * ct.least_g < kFaint)) {   // p may grow where the weights do not
#pragma unroll
                for (int h = 0; h < kH; ++h) over |= e[h] > kMostY;
            }
            uint32_t hmax = 0u, word[TERMS][2];
            uint32_t rest[kH / 2];
            const f32x2 vs2 = pack2(vs, vs);
#pragma unroll
            for (int h = 0; h < kH / 2; ++h) {
                e[2 * h] = ex2(e[2 * h]);
                e[2 * h + 1] = ex2(e[2 * h + 1]);
                const f32x2 w2 = mul2(mul2(pack2(e[2 * h], e[2 * h + 1]), vs2), reinterpret_cast<const f32x2 *>(ct.g + h0)[h]);
                float w0, w1;
                unpack2(w2, w0, w1);
                const uint32_t h2 = to_h2(w0, w1);
                hmax = h2_max(hmax, h2);
                uint16_t t[TERMS];
                rest[h] = split_weights<TERMS>(w0, w1, h2, t);
#pragma unroll
                for (int u = 0; u < TERMS; ++u) {
                    if (h & 1) word[u][h >> 1] |= (uint32_t)t[u] << 16;
                    else word[u][h >> 1] = t[u];
                }
            }
#pragma unroll
            for (int u = 0; u < TERMS; ++u)
                *reinterpret_cast<uint2 *>(sP + u * L::kTermP + row * kG + h0) = make_uint2(word[u][0], word[u][1]);
            over = !renew && (over || h2_lo(hmax) > kMostWeight || h2_hi(hmax) > kMostWeight);
            fence_proxy_async();   // the weights are read by the tensor core
            tmem_wait_st();
            tc_fence_before();
            if (!__syncthreads_or(over)) {
                if (TERMS == 2)
#pragma unroll
                    for (int h = 0; h < kH / 2; ++h) left[h] = h2_add(left[h], rest[h]);
                break;
            }
            renew = true;
        }
        const f32x2 vm2 = pack2(vm, vm);
#pragma unroll
        for (int h = 0; h < kH / 2; ++h) {
            const f32x2 e2 = pack2(e[2 * h], e[2 * h + 1]);
            l[h] = add2(l[h], e2);
            mv[h] = fma2(e2, vm2, mv[h]);
        }
        if (W) {   // two warps per block and head half: their sum does not depend on which comes first
            const float w = warp_sum8(e, lane);
            if ((lane & 3) == 0 && 2 * i + half < nloc) atomicAdd(&ct.w[2 * i + half][h0 + (lane >> 2)], w);
        }
    }

    // ---- sums over the token lanes
    {
        float x[3][kH];
#pragma unroll
        for (int h = 0; h < kH / 2; ++h) {
            unpack2(l[h], x[0][2 * h], x[0][2 * h + 1]);
            unpack2(mv[h], x[1][2 * h], x[1][2 * h + 1]);
            x[2][2 * h] = h2_lo(left[h]);
            x[2][2 * h + 1] = h2_hi(left[h]);
        }
        work_barrier();   // every thread has read ct.red
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            if (j == 2 && TERMS == 3) break;
            const float sum = warp_sum8(x[j], lane);
            if ((lane & 3) == 0) ct.red[j][warp & 3][h0 + (lane >> 2)] = __float_as_uint(sum);
        }
        work_barrier();
        if (tid < 3 * kG) {
            const int j = tid / kG, h = tid % kG;
            float sum = 0.0f;
            if (j < 2 || TERMS == 2)
                for (int w = 0; w < 4; ++w) sum += __uint_as_float(ct.red[j][w][h]);
            ct.sum[j][h] = sum;
        }
    }
    }
    __syncthreads();
    const size_t head0 = (size_t)qi * a.n_heads + (size_t)g * group;
    auto put = [&](int h, int d, float x) {
        const size_t at = (head0 + h) * kQDim + d;
        if (a.out_dt == QSA_F32) static_cast<float *>(a.out)[at] = x;
        else static_cast<uint16_t *>(a.out)[at] = (uint16_t)QFmt<F16>::bits(x);
    };
    float *part = reinterpret_cast<float *>(ring);   // split: this CTA's unnormalised output [16][128]
    if (warp == 8) {
    } else if (tl > 0) {
        wait_all(&ct.obar, (uint32_t)(tl - 1) & 1u, abort_flag);
        tc_fence_after();
        uint32_t o[2][kH];
#pragma unroll
        for (int u = 0; u < 2; ++u) tmem_ld8_nowait(tmem + lanes + L::kColO + u * kG + h0, o[u]);
        tmem_wait_ld();
        reg_fence(o[0]);
        reg_fence(o[1]);
        // this thread's dimension of its heads (a warp's stores for one head are 32 neighbours).  The codes'
        // mean, 7.5, times what the rounding left of the weights takes most of its effect away.
#pragma unroll
        for (int j = 0; j < kH; ++j) {
            const int h = h0 + j;
            float x = fmaf(__uint_as_float(o[1][j]), 0.0625f, __uint_as_float(o[0][j]));
            x = fmaf(fmaf(x, 512.0f, (7.5f / 16.0f) * ct.sum[2][h]), exp2f(-ct.eg[h]), ct.sum[1][h]);
            if (split > 1) part[h * kQDim + row] = x;
            else if (h < group) put(h, row, x / ct.sum[0][h]);
        }
        tc_fence_before();
    } else if (split == 1) {   // no visible token: o = 0
        for (int h = h0; h < min(group, h0 + kH); ++h) put(h, row, 0.0f);
    }
    if (tid == 0 && ct.abort) {   // a wait gave up: let what is in flight land before the memory is freed
        for (int i = max(0, tl - kStages); i < tl; ++i) mbar_drain(&ct.full[i % kStages], (uint32_t)(i / kStages) & 1u);
        for (int i = max(0, tl - 2); i < tl; ++i) mbar_drain(&ct.sbar[i & 1], (uint32_t)(i >> 1) & 1u);
        mbar_drain(&ct.obar, (uint32_t)(tl - 1) & 1u);
        if (a.flags) atomicOr(a.flags, QSA_FLAG_WAIT_TIMEOUT);
    }
    if (split == 1) {
        if (a.lse && tid < group)
            a.lse[head0 + tid] = tl > 0 ? (log2f(ct.sum[0][tid]) - ct.nm[tid]) * 0.6931471805599453f : -INFINITY;
        if (W && tid < nloc) {
            float w = 0.0f;
            for (int h = 0; h < group; ++h) w += ct.w[tid][h] / ct.sum[0][h];
            a.weights[((size_t)qi * a.n_kv_heads + g) * a.k + ct.slot[tid]] = w;
        }
    }
    __syncthreads();
    if (warp == 8) {
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
            st_cluster(&ct.ml[rank][h], x / kG, make_float2(tl > 0 ? -ct.nm[h] : none, tl > 0 ? ct.sum[0][h] : 0.0f));
        }
        cluster_sync();
        for (int hh = wg; wg < 2 && hh < nh; hh += 2) {
            const int h = rank * nh + hh;
            float M = -INFINITY, Lsum = 0.0f, acc = 0.0f;
            for (int r = 0; r < split; ++r)
                if (ct.ml[r][h].y != 0.0f) M = fmaxf(M, ct.ml[r][h].x);
            for (int r = 0; r < split; ++r) {
                const float2 v = ct.ml[r][h];
                if (v.y != 0.0f) {   // a CTA without tiles took no part
                    const float f = exp2f(v.x - M);
                    Lsum = fmaf(f, v.y, Lsum);
                    acc = fmaf(f, recv[(r * nh + hh) * kQDim + row], acc);
                }
            }
            if (h < group) {
                put(h, row, Lsum != 0.0f ? acc / Lsum : 0.0f);
                if (a.lse && row == 0) a.lse[head0 + h] = Lsum != 0.0f ? (M + log2f(Lsum)) * 0.6931471805599453f : -INFINITY;
            }
        }
        if (W) {
            if (tid < kG) {   // this CTA's part of the total, per head
                float M = -INFINITY, Lsum = 0.0f;
                for (int r = 0; r < split; ++r)
                    if (ct.ml[r][tid].y != 0.0f) M = fmaxf(M, ct.ml[r][tid].x);
                for (int r = 0; r < split; ++r)
                    if (ct.ml[r][tid].y != 0.0f) Lsum = fmaf(exp2f(ct.ml[r][tid].x - M), ct.ml[r][tid].y, Lsum);
                ct.fl[tid] = tl > 0 ? exp2f(-ct.nm[tid] - M) / Lsum : 0.0f;
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
