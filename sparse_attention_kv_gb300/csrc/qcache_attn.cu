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
// them are exact.  The other operands are split into e4m3 terms of 4 significant bits:
//   queries, scaled by a power of two per head: t0 + t1 (+ t2), stacked along K into one accumulator: two
//     terms hold a bf16 query (8 bits) exactly, three an fp16 one (11 bits), but for what lies below 2^-18 of
//     the head's largest value; in fp16, where that is more of them, its sum goes back times the mean code
//     (error of lse over single blocks 1.7e-6 of its norm without);
//   weights w = p vs g: t0 + (t1 + t2) / 16 with the second group in accumulator columns of its own,
//     two terms beside bf16 rows (2^-8 of the weight, as a bf16 weight would be), three beside fp16
//     (2^-12), with steps of 2^-18 of the largest weight at the small end.  The codes are not
//     centred, so a weight's rounding would count 7.5 steps too often: beside bf16 rows, what the two terms
//     leave of the weight's fp16 form (2^-11 of it; that rounding stays) is summed per head and goes back times
//     the mean code at the end.  Each remainder is exact, their fp16 sum good to 2^-11 of itself per token.  Error of the
//     output against fp64, 256 queries x 520,000 tokens: 0.0019 of its norm with it, 0.0025 without,
//     0.0017 from rounding the output to bf16 alone.
//
// A CTA takes (query, KV head) units in turn, two CTAs per SM; a step of it is four blocks, as two
// tiles of 128 rows: row 32q + r of tile s is block q's token 32s + r, so a thread's two tokens
// belong to one block.  Its warps:
//   0-7    softmax, two threads per row, eight heads each (in groups of up to eight heads one thread per row):
//          y = log2(e) s - m from S, p = 2^y, the weights' terms to shared memory (16 heads in a row per
//          token: B, MN-major), a block's sums of p;
//   8-11   unpacking, a row per thread: K's tokens and V^T's dimensions (the record holds V by
//          dimension) from shared into tensor memory, and the tokens' pairs to where the softmax reads them;
//   12     control: S = K . Q^T of step t + 1 as soon as its K is unpacked (M = 128 tokens, N = 16 heads, K = 128
//          dims x terms, A from tensor memory), then O += V^T . P^T of step t (M = 128 dims, K = 256 tokens);
//   13     preparation of the next unit: its distinct ids, and its queries' terms and sums (the first unit's
//          queries are shared out among the softmax warps: one warp takes 3 us for them);
//   14, 15 the record halves' copies, two steps deep, across units: K and all pairs, V.
// So K of the next step (of the next unit, too) unpacks and multiplies behind the softmax of this
// one, and nothing of a unit's start waits for memory but the first unit's.
// The references are lazy.  m[h] and the weights' scale g[h] (a power of two that puts the largest
// p vs seen at 2^4) are taken from a unit's first step, and change only when a later weight
// would pass 2^8 or its y 30: the barrier before O's product carries that vote, so an ordinary step
// has one wait and one barrier and no reduction across threads.  Sums of p (in fp32) stay per
// token lane until the unit's end.
//
// When units are few, a cluster of 2, 4 or 8 CTAs splits a unit's steps and combines the partial
// outputs through distributed shared memory.  Every wait is bounded; on expiry the CTA raises
// QSA_FLAG_WAIT_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
//
// Measured (device time in a graph of back-to-back calls, 256 queries x 64 heads in 4 groups x 520,000 tokens,
// k = 32, weights wanted): 62.6 us (fp16 69), where one read of each selected block by each query is 285 MB (42 us
// at the copy rate) and DRAM moves 218 MB; the 16-bit attention of the same selection takes 164 us.  It is
// bound by the softmax warps' chain of instructions (of a unit's 36,000 cycles, in a build that reads the clock:
// 1,800 until it stands prepared, 6,300 for the first step with its maxima, 3,400 for each other one, 4,200
// for the end; one CTA per SM takes 83 us), not by memory, tensor cores (12% busy) or the copies.  Without the
// weights 56 us (fp16 63).  Forms on the way, same call: one warpgroup doing everything 105 us; two sharing the heads,
// four CTAs per SM, 99; a control warp and S in two buffers, three CTAs per SM, 90; shared memory addressed as
// such 78.5; this division of labour 70; pairs through shared memory, float reductions 67.5; the first unit's
// queries shared out 64.  Not kept: reading S before the step's pairs or before the last step's end (74 and 79:
// outstanding tensor-memory loads hold up what follows), the unit's end in the unpacking warps (72), longer sleeps
// in the waits (no change), 88 registers for the softmax (no change), references made by every warp for itself
// (-2% in bf16, +2% in fp16 and in groups of eight).  At 80 registers a softmax thread the fp16 forms spill 116-124
// bytes, the bf16 ones 4-16.
#include <cuda.h>

#include <cmath>
#include <mutex>

#include "qcache.cuh"
#include "qsa_device.cuh"
#include "tc_ptx_tmem.cuh"

namespace qsa {
namespace {

constexpr int kG = 16;                    // head columns of a unit (heads past the group are zeros)
constexpr int kH = 8;                     // heads of a thread: two warpgroups share the 16
constexpr int kSel = QSA_ATTN_MAX_K;
constexpr int kWork = 256;                // threads of the two warpgroups
constexpr int kThreads = 512;             // and a warpgroup that unpacks, and one of single warps
constexpr int kUnpack = 8, kControl = 12, kPrepare = 13, kFetch = 14;   // first warps of the roles
constexpr int kStep = 4;                  // blocks of a step
constexpr int kKBytes = kQOffV, kVBytes = kQRec - kQOffV;  // a record's halves: K codes and all pairs, V codes
constexpr int kVStages = 2;
constexpr int kMaxSplit = 8;
constexpr float kTop = 4.0f;              // log2 of the largest weight when the references are set
// (a weight whose leading term is 256 or more moves them; e4m3 holds 448)
constexpr float kMostY = 30.0f;           // and a y above this
constexpr float kFaint = 0x1p-60f;        // V scales whose weights may stay small until p overflows

// What the preparation warp leaves of a unit.
struct QUnit {
    int steps;                            // of this CTA's slice; 0: no visible token
    int b0, nloc;                         // first entry and length of the slice of sel
    int ntok;
    int32_t sel[kSel + kStep];            // the distinct valid ids, in slot order, then ids past every context
    int32_t slot[kSel];                   // and the slots they came from
    alignas(16) float f[kG];              // scale log2(e) 2^9 / (the head's power-of-two scaling of q)
    alignas(16) float qs[kG];             // scale log2(e) sum(q)
    alignas(16) float fc[kG];             // f times what the terms left of the queries times the codes' mean, 7.5 (fp16)
};

struct QCtrl {
    uint64_t k_full[2], k_free[2], v_full[kVStages], v_free[kVStages], sbar[2], obar;
    uint64_t ids_ready[2], ready[2], done[2], drained;
    uint32_t tmem_base;
    int abort;
    QUnit unit[2];
    // a step's pairs (K, V) by tile and row; a V scale of -1: not seen.  Three steps: those of t + 1 are written while
    // a slow warp may still read those of t - 1
    alignas(16) uint2 token[3][kStep * kQBlockTok];
    alignas(16) float zero[kG];
    alignas(16) float nm[kG];             // minus the reference of the exponents (log2 units)
    alignas(16) float g[kG];              // power of two of the weights
    alignas(16) float fl[kG];             // rescaling of the sums and of the outputs
    alignas(16) float fo[kG];
    float top[kG], eg[kG];                // largest log2(p vs) + m seen, log2(g)
    float ig[kG];                         // 1 / g
    float least_g;
    float red[2][4][kG];                  // maxima by warp
    float part[3][4][kG];                 // a unit's sums by warp: l, sum of p vm, 16 x what the weights' rounding took away
    alignas(16) float fin[8][4][kG];      // a warp's copy of the heads' factors of the outputs, and 1 / l
    float sum[kG];                        // l
    float2 ml[kMaxSplit][kG];             // (m, l) of every CTA of a cluster
    alignas(16) float w[kSel][kG];        // sums of p over a slot's tokens
};

template <int TERMS>
struct QLayout {
    static constexpr int kQBytes = kG * TERMS * 128;             // heads x terms rows of 128 bytes, swizzled
    static constexpr int kTermP = 128 * kG;                      // [128 tokens][16 heads]
    static constexpr int kTileP = TERMS * kTermP;
    static constexpr int kOffQ = 0;                              // two units' queries
    static constexpr int kOffP = kOffQ + 2 * kQBytes;
    static constexpr int kStepP = 2 * kTileP;                    // the two tiles of a step
    static constexpr int kPBufs = TERMS == 2 ? 2 : 1;            // what the shared memory of two CTAs holds
    static constexpr int kKStages = 2;
    static constexpr int kOffK = kOffP + kPBufs * kStepP;
    static constexpr int kOffV = kOffK + kKStages * kStep * kKBytes;
    static constexpr int kOffCtrl = kOffV + kVStages * kStep * kVBytes;
    static constexpr int kBytes = kOffCtrl + (int)sizeof(QCtrl) + 1024;   // + alignment slack
};
// tensor memory: S (two steps of two tiles), O (two groups of columns: the leading terms, and the
// others 16 times as large), the unpacked K tiles and the unpacked V tiles
constexpr uint32_t kColS = 0, kColO = 64, kColK = 96, kColV = 160, kCols = 256;
// two CTAs (and 1 KB each that the system keeps) in an SM's 228 KB
static_assert(2 * (QLayout<2>::kBytes + 1024) <= 228 * 1024 && 2 * (QLayout<3>::kBytes + 1024) <= 228 * 1024, "two CTAs per SM");
// the combine's buffers fit the ring: outputs sent and received, 16 heads x 128 fp32 each
static_assert(2 * kG * kQDim * 4 <= 2 * kStep * kKBytes, "combine buffers");

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
// Two fp32 values to fp16 (b high), two fp16 pairs (or four fp32 values) to four e4m3 and back (exact).
__device__ __forceinline__ uint32_t to_h2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t h4_to_e4m3(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 y, %2;\n\t"
        "mov.b32 %0, {x, y};\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t f4_to_e4m3(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\t"
        "mov.b32 %0, {x, y};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
__device__ __forceinline__ void e4m3_to_h4(uint32_t e, uint32_t &a, uint32_t &b) {
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(e));
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
// The warp's largest value (a NaN counts as none).
__device__ __forceinline__ float warp_fmax(float x) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float h2_lo(uint32_t h) { return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu))); }
__device__ __forceinline__ float h2_hi(uint32_t h) { return __half2float(__ushort_as_half((unsigned short)(h >> 16))); }
constexpr uint32_t kH16 = 0x4C004C00u, kHNeg16 = 0xCC00CC00u;   // (16, 16) and (-16, -16)

// The e4m3 terms of four weights, at most 448: w = t0 + (t1 + t2) / 16 + what is left.  Two terms: from the
// fp16 pairs h, whose 11 bits are more than theirs; what is left of h, 16 times as large, is exact, and added to `left`
// in fp16.
template <int TERMS>
__device__ __forceinline__ void split_weights(const float (&w)[4], const uint32_t (&h)[2], uint32_t (&t)[TERMS],
                                              uint32_t (&left)[2]) {
    uint32_t a, b;
    if constexpr (TERMS == 2) {
        t[0] = h4_to_e4m3(h[0], h[1]);
        e4m3_to_h4(t[0], a, b);
        const uint32_t r0 = h2_fma(a, kHNeg16, h2_mul(h[0], kH16)), r1 = h2_fma(b, kHNeg16, h2_mul(h[1], kH16));
        t[1] = h4_to_e4m3(r0, r1);
        e4m3_to_h4(t[1], a, b);
        left[0] = h2_add(left[0], h2_sub(r0, a));
        left[1] = h2_add(left[1], h2_sub(r1, b));
    } else {   // the first remainders in fp32; they fit fp16 with bits to spare
        t[0] = f4_to_e4m3(w[0], w[1], w[2], w[3]);
        e4m3_to_h4(t[0], a, b);
        const uint32_t r0 = to_h2((w[0] - h2_lo(a)) * 16.0f, (w[1] - h2_hi(a)) * 16.0f);
        const uint32_t r1 = to_h2((w[2] - h2_lo(b)) * 16.0f, (w[3] - h2_hi(b)) * 16.0f);
        t[1] = h4_to_e4m3(r0, r1);
        e4m3_to_h4(t[1], a, b);
        t[2] = h4_to_e4m3(h2_sub(r0, a), h2_sub(r1, b));
    }
}
// The e4m3 terms of four query values below 256: v = t0 + t1 (+ t2), exact for the format's significand down
// to 2^-10 (bf16) and 2^-7 (fp16) of the head's largest value, to 2^-18 of it below.
// What is left stays in h0 and h1.
template <int TERMS>
__device__ __forceinline__ void split_query(uint32_t &h0, uint32_t &h1, uint32_t (&t)[TERMS]) {
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
        uint32_t a, b;
        t[u] = h4_to_e4m3(h0, h1);
        e4m3_to_h4(t[u], a, b);
        h0 = h2_sub(h0, a);
        h1 = h2_sub(h1, b);
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


// Every thread of the warp waits, a bounded number of tries: one that fails suspends the thread for 3.9 us (measured on
// a barrier that nobody arrives at, with and without the sleeps), so 2^18 come to a second.  After one wait has given
// up, waits for copies and products return at once, and the CTA runs through its remaining steps without their results.
// Waits for what another warp does (HANDSHAKE) go on and have four times as many, so that one that began before the wait
// that gave up does not run out while the other warp still waits: every warp makes its steps, and all of them read
// the same number of steps, so that the barriers meet.  (A look at the clock in the loop, as the other kernels' waits
// take, made the deep prompt's call 5% slower: the waits' code stands in the loop of every role.)
template <int SLEEP = 0, bool HANDSHAKE = false>
__device__ __forceinline__ void wait_all(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (__all_sync(kFull, ok != 0)) return;   // the warp stays converged
    const uint32_t most = HANDSHAKE ? 1u << 20 : *abort_flag ? 1u : 1u << 18;
    if constexpr (SLEEP == 0)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n\t"
            "WAIT_%=:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE_%=;\n\t"
            "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, %3;\n\t@q bra WAIT_%=;\n\tDONE_%=:\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(most)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n\t"
            "WAIT_%=:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE_%=;\n\t"
            "nanosleep.u32 %4;\n\t"
            "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, %3;\n\t@q bra WAIT_%=;\n\tDONE_%=:\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(most), "n"(SLEEP)
            : "memory");
    if (!ok) *abort_flag = 1;
    __syncwarp();
}

// Barriers: 1 among the softmax warps, 2 and 4 from the unpacking warps to the control warp (K and V stand),
// 3 with a vote among the softmax warps and the control warp.
__device__ __forceinline__ void work_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void k_ready_arrive() { asm volatile("bar.arrive 2, 160;" ::: "memory"); }
__device__ __forceinline__ void k_ready_wait() { asm volatile("bar.sync 2, 160;" ::: "memory"); }
__device__ __forceinline__ void v_ready_arrive() { asm volatile("bar.arrive 4, 160;" ::: "memory"); }
__device__ __forceinline__ void v_ready_wait() { asm volatile("bar.sync 4, 160;" ::: "memory"); }
__device__ __forceinline__ bool vote_barrier(bool mine) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 3, 288, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)mine)
        : "memory");
    return any != 0;
}
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
// 2^x for an integer x in [-126, 127].
__device__ __forceinline__ float pow2i(int x) { return __int_as_float((x + 127) << 23); }

struct QParams {
    QAttnArgs a;
    float scale_log2;
    int split;
    int units;
};

// The preparation warp: a unit's distinct ids inside its context, in slot order, and this CTA's slice of them.
template <bool W>
__device__ __forceinline__ void prepare_ids(const QParams &p, int qi, int g, int rank, QUnit &u) {
    const QAttnArgs &a = p.a;
    const int lane = threadIdx.x & 31;
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
        u.sel[at] = r0;
        u.slot[at] = lane;
    }
    if (take1) {
        const int at = __popc(m0) + __popc(m1 & below);
        u.sel[at] = r1;
        u.slot[at] = lane + 32;
    }
    if (lane < kStep) u.sel[nsel + lane] = QSA_MAX_BLOCKS;
    const bool any_bad = __any_sync(kFull, bad);
    if (lane == 0) {
        const int T = (nsel + kStep - 1) / kStep, p0 = rank * T / p.split, p1 = (rank + 1) * T / p.split;   // slices of whole steps
        u.b0 = kStep * p0;
        u.nloc = min(nsel, kStep * p1) - kStep * p0;
        u.steps = p1 - p0;
        u.ntok = ntok;
        if (any_bad && g == 0 && rank == 0 && a.flags) atomicOr(a.flags, QSA_FLAG_BAD_ID);
    }
    if (W && rank == 0) {   // slots that take no part
        float *w = a.weights + ((size_t)qi * a.n_kv_heads + g) * a.k;
        if (lane < a.k && !take0) w[lane] = 0.0f;
        if (lane + 32 < a.k && !take1) w[lane + 32] = 0.0f;
    }
}

// One warp: N (2 or 8) of the group's queries from head hh, as e4m3 terms (four dimensions of a head per lane).
template <bool F16, int TERMS, int N>
__device__ __forceinline__ void prepare_queries(const QParams &p, int u_at, int group, int hh, QUnit &u, uint8_t *sQ) {
    const QAttnArgs &a = p.a;
    const int lane = threadIdx.x & 31, qi = u_at / a.n_kv_heads, g = u_at - qi * a.n_kv_heads;
    const uint16_t *q = static_cast<const uint16_t *>(a.qa) + qi * a.q_stride + (int64_t)(g * group) * a.q_head_stride + lane * 4;
    uint2 raw[N];
#pragma unroll
    for (int j = 0; j < N; ++j)
        raw[j] = hh + j < group ? *reinterpret_cast<const uint2 *>(q + (hh + j) * a.q_head_stride) : make_uint2(0u, 0u);
    float sums[N], lefts[N];
    int es[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int h = hh + j;
        const float x[4] = {QFmt<F16>::lo(raw[j].x), QFmt<F16>::hi(raw[j].x), QFmt<F16>::lo(raw[j].y), QFmt<F16>::hi(raw[j].y)};
        uint32_t big = 0u;   // the bits of the largest magnitude (an infinity or a NaN stays the largest)
#pragma unroll
        for (int i = 0; i < 4; ++i) big = max(big, __float_as_uint(x[i]) & 0x7FFFFFFFu);
        big = __reduce_max_sync(kFull, big);
        sums[j] = (x[0] + x[1]) + (x[2] + x[3]);
        const bool finite = big < 0x7F800000u;
        // a power of two that puts the largest magnitude into [128, 256), in two exact steps
        const int lg = big >= 0x00800000u ? (int)(big >> 23) - 127 : -118 - __clz((int)big);
        const int e = finite && big != 0u ? 7 - lg : 0;
        es[j] = finite ? e : 1024;
        const float s0 = pow2i(e >> 1), s1 = pow2i(e - (e >> 1));
        uint32_t terms[TERMS];
        uint32_t h0 = finite ? to_h2(x[0] * s0 * s1, x[1] * s0 * s1) : 0u;
        uint32_t h1 = finite ? to_h2(x[2] * s0 * s1, x[3] * s0 * s1) : 0u;
        split_query<TERMS>(h0, h1, terms);
        if (F16) lefts[j] = (h2_lo(h0) + h2_hi(h0)) + (h2_lo(h1) + h2_hi(h1));
#pragma unroll
        for (int t = 0; t < TERMS; ++t)
            *reinterpret_cast<uint32_t *>(sQ + (t * kG + h) * 128 + (((lane >> 2) ^ (h & 7)) << 4) + (lane & 3) * 4) = terms[t];
    }
    constexpr int kPer = 32 / N;   // lanes that hold a head's sum
    auto over_lanes = [&](float (&x)[N]) {
        if constexpr (N == 8) {
            return warp_sum8(x, lane);
        } else {                   // the same pairs in the same order
            static_assert(N == 2, "two or eight heads");
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                x[0] += __shfl_xor_sync(kFull, x[0], o);
                x[1] += __shfl_xor_sync(kFull, x[1], o);
            }
            return lane < kPer ? x[0] : x[1];
        }
    };
    const float sum = over_lanes(sums), left = F16 ? over_lanes(lefts) : 0.0f;
    int e = es[0];
#pragma unroll
    for (int j = 1; j < N; ++j) e = lane / kPer == j ? es[j] : e;
    if (lane % kPer == 0) {
        const int h = hh + lane / kPer;
        const float f = e == 1024 ? __uint_as_float(0x7FC00000u) : scalbnf(p.scale_log2, 9 - e);
        u.f[h] = f;
        if (F16) u.fc[h] = f * (left * (7.5f / 512.0f));
        u.qs[h] = p.scale_log2 * sum;
    }
}

// F16: rows and queries in fp16 (three terms), otherwise bf16 (two); W: the slots' weights are wanted; HALF: groups
// of at most eight heads, whose softmax threads take one token and eight heads each instead of two tokens and half
// of sixteen heads (256 queries x 8 KV heads x 8 heads, k = 32: 100 us, by the form for sixteen 122; in fp16 107
// and 134; one query 7.8 and 8.1.  One warpgroup for eight heads and the other idle took 115 where this took 101).
template <bool F16, bool W, bool HALF>
__global__ void __launch_bounds__(kThreads, 2) qattn_kernel(const __grid_constant__ QParams p) {
    constexpr int TERMS = F16 ? 3 : 2;
    using L = QLayout<TERMS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem + L::kOffQ, *sP = smem + L::kOffP, *sK = smem + L::kOffK, *sV = smem + L::kOffV;
    QCtrl &ct = *reinterpret_cast<QCtrl *>(smem + L::kOffCtrl);
    volatile int *abort_flag = &ct.abort;
    const QAttnArgs &a = p.a;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const int split = p.split, rank = split > 1 ? (int)cluster_ctarank() : 0;
    const int u0 = blockIdx.x / split, ustep = gridDim.x / split;
    const int group = a.n_heads / a.n_kv_heads, nb_cap = a.capacity / kQBlockTok;

    for (int i = tid; i < (int)(sizeof(QCtrl) / 4); i += kThreads) reinterpret_cast<uint32_t *>(&ct)[i] = 0u;
    __syncthreads();
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ct.k_full[i], 1);
            mbar_init(&ct.k_free[i], 4);  // the unpacking warps
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&ct.v_full[i], 1);
            mbar_init(&ct.v_free[i], 4);  // the unpacking warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ct.sbar[i], 5);    // S is complete, and the unpacking warps' pairs stand
            mbar_init(&ct.ids_ready[i], 1);
            mbar_init(&ct.ready[i], 2);   // the ids, the queries
            mbar_init(&ct.done[i], 15);   // all warps but the preparing one
        }
        mbar_init(&ct.obar, 1);
        mbar_init(&ct.drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    // a programmatic dependent of the work before it: nothing is read, and no tensor memory taken,
    // before that work is complete
    wait_prior_grid();
    __syncwarp();

    // Every role walks the same units (n-th unit u, buffer n & 1) and the same steps (t-th step, stage t & 1).
    int stage = 0;                        // a copying warp's next stage, and how often it has filled the last one
    uint32_t lap = 0;
    if (warp >= kControl) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kPrepare) {
        for (int u = u0, n = 0; u < p.units; u += ustep, ++n) {
            if (n >= 2) wait_all<256, true>(&ct.done[n & 1], ((uint32_t)(n >> 1) - 1u) & 1u, abort_flag);
            const int qi = u / a.n_kv_heads, g = u - qi * a.n_kv_heads;
            prepare_ids<W>(p, qi, g, rank, ct.unit[n & 1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&ct.ids_ready[n & 1]);
            if (n > 0)   // the first unit's queries come from the softmax warps
#pragma unroll 1
                for (int hh = 0; hh < kG; hh += 8)
                    prepare_queries<F16, TERMS, 8>(p, u, group, hh, ct.unit[n & 1], sQ + (n & 1) * L::kQBytes);
            fence_proxy_async();   // the queries are read by the tensor core
            __syncwarp();
            if (lane < (n > 0 ? 2 : 1)) mbar_arrive(&ct.ready[n & 1]);
        }
    } else if (warp >= kFetch) {
        // copies, a lane per block: the first warp K and the pairs, the second V
        const bool is_k = warp == kFetch;
        static_assert(L::kKStages == 2 && kVStages == 2, "two stages each");
        const uint32_t bytes = is_k ? kKBytes : kVBytes;
        uint64_t *full = is_k ? ct.k_full : ct.v_full, *vacant = is_k ? ct.k_free : ct.v_free;
        for (int u = u0, n = 0; u < p.units; u += ustep, ++n) {
            wait_all<64, true>(&ct.ids_ready[n & 1], (uint32_t)(n >> 1) & 1u, abort_flag);
            const QUnit &un = ct.unit[n & 1];
            const int steps = un.steps, nloc = un.nloc;
            const uint8_t *head = static_cast<const uint8_t *>(a.cache) + qrec_offset(u % a.n_kv_heads, nb_cap, 0) + (is_k ? 0 : kQOffV);
            for (int i = 0; i < steps; ++i) {
                const int m = min(kStep, nloc - kStep * i);
                const uint8_t *src = head + (size_t)un.sel[un.b0 + kStep * i + min(lane, m - 1)] * kQRec;
                if (lap > 0) wait_all<32>(&vacant[stage], (lap - 1u) & 1u, abort_flag);
                if (__any_sync(kFull, *abort_flag != 0)) break;   // the stage may still be in use
                if (lane == 0) mbar_expect_tx(&full[stage], (uint32_t)m * bytes);
                __syncwarp();
                if (lane < m) bulk_load((is_k ? sK : sV) + (stage * kStep + lane) * bytes, src, bytes, &full[stage]);
                __syncwarp();
                if (++stage == 2) {
                    stage = 0;
                    ++lap;
                }
            }
            if (lane == 0) mbar_arrive(&ct.done[n & 1]);
            __syncwarp();
        }
    } else if (warp == kControl) {
        tmem_alloc(&ct.tmem_base, kCols);
        tmem_relinquish();
    }
    if (warp < kUnpack) {   // nothing to do yet: two heads of the first unit's queries each
        prepare_queries<F16, TERMS, 2>(p, u0, group, 2 * warp, ct.unit[0], sQ);
        fence_proxy_async();
        work_barrier();
        if (tid == 0) mbar_arrive(&ct.ready[0]);
        __syncwarp();
    }
    if (warp <= kControl) {
    tc_fence_before();
    asm volatile("bar.sync 3, 416;" ::: "memory");   // the softmax, unpacking and control warps
    tc_fence_after();
    const uint32_t tmem = ct.tmem_base;
    if (warp == kControl) {
        const uint64_t dq = sdesc(smem_u32(sQ)), dp = sdesc_mn(smem_u32(sP), 8 * kG, L::kTermP);
        auto scores = [&](int n, int t) {   // step t, of unit n
            wait_all<0, true>(&ct.ready[n & 1], (uint32_t)(n >> 1) & 1u, abort_flag);
            k_ready_wait();
            tc_fence_after();
            if (elect_one()) {
                const uint64_t d = dq + (n & 1) * (L::kQBytes / 16);   // descriptors count in units of 16 bytes
                for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                    for (int x = 0; x < TERMS; ++x)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f8_ta(tmem + kColS + (t & 1) * 2 * kG + sub * kG, tmem + kColK + sub * 32 + kk * 8,
                                      d + x * (kG * 8) + kk * 2, idesc(0, 128, kG), (x | kk) != 0 ? 1u : 0u);
                mma_commit(&ct.sbar[t & 1]);
            }
            __syncwarp();
        };
        bool primed = false;
        for (int u = u0, n = 0, t = 0; u < p.units; u += ustep, ++n) {
            wait_all<0, true>(&ct.ids_ready[n & 1], (uint32_t)(n >> 1) & 1u, abort_flag);
            const int steps = ct.unit[n & 1].steps;
            if (steps == 0) primed = false;
            // i = -1: the first step's S, unless it was issued behind the last unit's last step
            for (int i = -1; i < steps; ++i) {
                int of = n;                                // the unit of the next S
                bool next = i < 0 ? steps > 0 && !primed : i + 1 < steps;
                if (i + 1 == steps && steps > 0 && u + ustep < p.units) {
                    of = n + 1;
                    wait_all<0, true>(&ct.ready[of & 1], (uint32_t)(of >> 1) & 1u, abort_flag);
                    next = ct.unit[of & 1].steps > 0;
                }
                if (i + 1 == steps) primed = next && of != n;
                if (next) scores(of, t + (i >= 0 ? 1 : 0));
                if (i < 0) continue;
                v_ready_wait();
                while (vote_barrier(false)) {}             // again while the references move
                tc_fence_after();
                if (elect_one()) {
                    for (int sub = 0; sub < 2; ++sub) {
                        const uint64_t d = dp + (t % L::kPBufs) * (L::kStepP / 16) + sub * (L::kTileP / 16);
                        const uint32_t v = tmem + kColV + sub * 32;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)   // both groups of columns
                            mma_f8_ta(tmem + kColO, v + kk * 8, d + kk * (2 * kG), idesc(0, 128, 2 * kG) | kIdescBMn,
                                      (i | sub | kk) != 0 ? 1u : 0u);
                        if (TERMS == 3)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_f8_ta(tmem + kColO + kG, v + kk * 8, d + 2 * (L::kTermP / 16) + kk * (2 * kG),
                                          idesc(0, 128, kG) | kIdescBMn, 1u);
                    }
                    mma_commit(&ct.obar);
                }
                __syncwarp();
                ++t;
            }
            if (lane == 0) mbar_arrive(&ct.done[n & 1]);
            __syncwarp();
        }
    } else if (warp >= kUnpack) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        // ---- unpacking: a row of A per thread, 32 bytes of codes at a time to 8 + 8 columns (low and high nibbles)
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int q = warp & 3, row = (q << 5) | lane;
        auto unpack = [&](const uint8_t *a0, const uint8_t *a1, uint32_t lo_col, uint32_t hi_col) {
            const uint4 x0 = *reinterpret_cast<const uint4 *>(a0), x1 = *reinterpret_cast<const uint4 *>(a1);
            const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            uint32_t lo[8], hi[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                lo[j] = w[j] & 0x0F0F0F0Fu;
                hi[j] = (w[j] >> 4) & 0x0F0F0F0Fu;
            }
            tmem_st8(tmem + lanes + lo_col, lo);
            tmem_st8(tmem + lanes + hi_col, hi);
        };
        // K of step t, step i of unit un: block q's tokens `lane` (tile 0) and 32 + `lane` (tile 1), their 128
        // dimensions and their pairs
        auto unpack_k = [&](int t, const QUnit &un, int i) {
            const int s = t % L::kKStages;
            wait_all<32>(&ct.k_full[s], (uint32_t)(t / L::kKStages) & 1u, abort_flag);
            tc_fence_after();
            const uint8_t *rec = sK + (s * kStep + q) * kKBytes;
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                constexpr int kPlane = kQBlockTok * 16;
                const uint8_t *src = rec + (32 * sub + lane) * 16;
                unpack(src, src + kPlane, kColK + sub * 32, kColK + sub * 32 + 16);
                unpack(src + 2 * kPlane, src + 3 * kPlane, kColK + sub * 32 + 8, kColK + sub * 32 + 24);
            }
            const int left = un.ntok - un.sel[un.b0 + kStep * i + q] * kQBlockTok;   // tokens of this block below the context's end
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                const uint32_t kp = *reinterpret_cast<const uint32_t *>(rec + kQOffKPair + (32 * sub + lane) * 4);
                const uint32_t vp = *reinterpret_cast<const uint32_t *>(rec + kQOffVPair + (32 * sub + lane) * 4);
                ct.token[t % 3][sub * 128 + row] = 32 * sub + lane < left ? make_uint2(kp, vp) : make_uint2(0u, F16 ? 0xBC00u : 0xBF80u);
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&ct.k_free[s]);   // the stores to tensor memory are fed from registers
                mbar_arrive(&ct.sbar[t & 1]);
            }
            __syncwarp();
            tmem_wait_st();
            tc_fence_before();
            k_ready_arrive();
        };
        bool primed = false;
        for (int u = u0, n = 0, t = 0; u < p.units; u += ustep, ++n) {
            wait_all<0, true>(&ct.ready[n & 1], (uint32_t)(n >> 1) & 1u, abort_flag);
            const int steps = ct.unit[n & 1].steps;
            if (steps == 0) primed = false;
            for (int i = -1; i < steps; ++i) {             // as the control warp walks
                int of = n;
                bool next = i < 0 ? steps > 0 && !primed : i + 1 < steps;
                if (i + 1 == steps && steps > 0 && u + ustep < p.units) {
                    of = n + 1;
                    wait_all<0, true>(&ct.ready[of & 1], (uint32_t)(of >> 1) & 1u, abort_flag);
                    next = ct.unit[of & 1].steps > 0;
                }
                if (i + 1 == steps) primed = next && of != n;
                if (i >= 0) wait_all<32>(&ct.sbar[t & 1], (uint32_t)(t >> 1) & 1u, abort_flag);   // K(t) is read
                if (next) unpack_k(t + (i >= 0 ? 1 : 0), ct.unit[of & 1], of == n ? i + 1 : 0);
                if (i < 0) continue;
                const int s = t % kVStages;
                wait_all(&ct.v_full[s], (uint32_t)(t / kVStages) & 1u, abort_flag);
                if (t > 0) wait_all<32>(&ct.obar, (uint32_t)(t - 1) & 1u, abort_flag);   // V(t - 1) is read
                tc_fence_after();
                // V: this thread's dimension; the blocks' tokens 0..31 are the low nibbles (tile 0)
                const uint8_t *src = sV + s * kStep * kVBytes + row * 16;
#pragma unroll
                for (int b = 0; b < kStep; ++b)
                    unpack(src + b * kVBytes, src + b * kVBytes + 2048, kColV + b * 8, kColV + 32 + b * 8);
                if (lane == 0) mbar_arrive(&ct.v_free[s]);   // the stores are fed from registers
                __syncwarp();
                tmem_wait_st();
                tc_fence_before();
                v_ready_arrive();
                ++t;
            }
            if (lane == 0) mbar_arrive(&ct.done[n & 1]);
            __syncwarp();
        }
    } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
    // ---- softmax: two threads per token pair, eight heads each.  Rows 32q .. 32q + 31 of both tiles are block
    // q's tokens 0..31 and 32..63, so a warp holds tokens of one block only.
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int wg = warp >> 2, q = warp & 3, row = tid & 127;
    // HALF: each warpgroup takes one tile's tokens and all (at most eight) heads, and sums of theirs go to columns
    // of its own; the weights of heads 8..15 stay 0
    constexpr int SUBS = HALF ? 1 : 2;
    constexpr int kHO = HALF ? kH / 2 : kH;                          // heads of a thread's outputs
    const int c0 = wg * kH, h0 = HALF ? 0 : c0, ho = HALF ? wg * kHO : c0, sub0 = HALF ? wg : 0;
    if (HALF && wg == 1) {
        for (int i = 0; i < L::kPBufs * 2 * TERMS; ++i)
            *reinterpret_cast<uint2 *>(sP + i * L::kTermP + row * kG + kH) = make_uint2(0u, 0u);
        fence_proxy_async();
    }
    for (int u = u0, n = 0, t = 0; u < p.units; u += ustep, ++n) {
        const QUnit &un = ct.unit[n & 1];
        wait_all<0, true>(&ct.ready[n & 1], (uint32_t)(n >> 1) & 1u, abort_flag);
        const int steps = un.steps, nloc = un.nloc;
        f32x2 l[kH / 2], mv[kH / 2];
        uint32_t left[kH / 2];            // fp16 pairs: 16 x what the rounding of this thread's weights left
#pragma unroll
        for (int h = 0; h < kH / 2; ++h) {
            l[h] = mv[h] = 0ull;
            left[h] = 0u;
        }
        for (int i = 0; i < steps; ++i, ++t) {
            // S(t) is complete; so is, two steps back, O += P(t - 2) V(t - 2), which the control warp issued before it
            wait_all(&ct.sbar[t & 1], (uint32_t)(t >> 1) & 1u, abort_flag);
            if (L::kPBufs == 1 && t > 0) wait_all(&ct.obar, (uint32_t)(t - 1) & 1u, abort_flag);   // P(t - 1) is read
            tc_fence_after();
            float ks[SUBS], km[SUBS], vs[SUBS], vm[SUBS];
#pragma unroll
            for (int sub = 0; sub < SUBS; ++sub) {
                const uint2 x = ct.token[t % 3][(sub0 + sub) * 128 + row];
                ks[sub] = QFmt<F16>::lo(x.x), km[sub] = QFmt<F16>::hi(x.x);
                vs[sub] = QFmt<F16>::lo(x.y), vm[sub] = QFmt<F16>::hi(x.y);
            }
            const bool all_vis = __all_sync(kFull, !(vs[SUBS - 1] < 0.0f));   // and so the first tile's
            // y = log2(e) s - m of this thread's tokens, into e
            float e[SUBS][kH];
            auto logits = [&](const float *nmp) {
                uint32_t v[SUBS][kH];
#pragma unroll
                for (int sub = 0; sub < SUBS; ++sub)
                    tmem_ld8_nowait(tmem + lanes + kColS + ((t & 1) * 2 + sub0 + sub) * kG + h0, v[sub]);
                tmem_wait_ld();
#pragma unroll
                for (int sub = 0; sub < SUBS; ++sub) reg_fence(v[sub]);
#pragma unroll
                for (int h = 0; h < kH / 2; h += 2) {
                    const ulonglong2 nm = *reinterpret_cast<const ulonglong2 *>(nmp + h0 + 2 * h);
                    const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(un.f + h0 + 2 * h);
                    const ulonglong2 qs = *reinterpret_cast<const ulonglong2 *>(un.qs + h0 + 2 * h);
                    ulonglong2 fc = make_ulonglong2(0ull, 0ull);
                    if (F16) fc = *reinterpret_cast<const ulonglong2 *>(un.fc + h0 + 2 * h);
#pragma unroll
                    for (int sub = 0; sub < SUBS; ++sub) {
                        const f32x2 ks2 = pack2(ks[sub], ks[sub]), km2 = pack2(km[sub], km[sub]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int x = 2 * (h + j);
                            const f32x2 s2 = pack2(__uint_as_float(v[sub][x]), __uint_as_float(v[sub][x + 1]));
                            const f32x2 sf = F16 ? fma2(s2, j ? f.y : f.x, j ? fc.y : fc.x) : mul2(s2, j ? f.y : f.x);
                            const f32x2 y = fma2(sf, ks2, fma2(km2, j ? qs.y : qs.x, j ? nm.y : nm.x));
                            unpack2(y, e[sub][x], e[sub][x + 1]);
                        }
                    }
                }
                if (!all_vis)
#pragma unroll
                    for (int sub = 0; sub < SUBS; ++sub)
#pragma unroll
                        for (int h = 0; h < kH; ++h) e[sub][h] = vs[sub] < 0.0f ? -INFINITY : e[sub][h];
            };
            int renew = i == 0 ? 1 : 0;       // 1: the references move before the weights are made; 2: they have
            while (true) {
                logits(i == 0 && renew == 1 ? ct.zero : ct.nm);
                if (renew == 1) {
                    // new references: the largest exponent and the largest weight so far, per head
                    float lv[SUBS];
#pragma unroll
                    for (int sub = 0; sub < SUBS; ++sub) lv[sub] = vs[sub] > 0.0f ? lg2(vs[sub]) : -INFINITY;
                    float mine[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int h = 0; h < kH; ++h) {
                        const float y = warp_fmax(HALF ? e[0][h] : fmaxf(e[0][h], e[SUBS - 1][h]));
                        const float r = warp_fmax(HALF ? e[0][h] + lv[0] : fmaxf(e[0][h] + lv[0], e[SUBS - 1][h] + lv[SUBS - 1]));
                        if (lane == h) {
                            mine[0] = y;
                            mine[1] = r;
                        }
                    }
                    if (lane < kH) {
                        ct.red[0][warp & 3][c0 + lane] = mine[0];
                        ct.red[1][warp & 3][c0 + lane] = mine[1];
                    }
                    work_barrier();
                    if (warp == 0) {
                        const int h = lane & 15;
                        float y = -INFINITY, r = -INFINITY;
                        for (int w = 0; w < 4; ++w) {
                            y = fmaxf(y, ct.red[0][w][h]);
                            r = fmaxf(r, ct.red[1][w][h]);
                        }
                        if (HALF) {   // both tiles' tokens
                            y = fmaxf(y, __shfl_xor_sync(kFull, y, kH));
                            r = fmaxf(r, __shfl_xor_sync(kFull, r, kH));
                        }
                        const float m0 = i == 0 ? 0.0f : -ct.nm[h], rise = y;
                        const float m1 = i == 0 ? rise : m0 + fmaxf(rise, 0.0f);
                        const float top = fmaxf(i == 0 ? -INFINITY : ct.top[h], m0 + r);
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
                            ct.ig[h] = exp2f(-eg);
                            if (lane == 0) ct.least_g = exp2f(least);
                        }
                    }
                    work_barrier();
                    if (i > 0) {   // what is summed so far, to the new references
                        wait_all(&ct.obar, (uint32_t)(t - 1) & 1u, abort_flag);   // O(t - 1) is complete
                        tc_fence_after();
#pragma unroll
                        for (int h = 0; h < kH / 2; ++h) {
                            const f32x2 fl = reinterpret_cast<const f32x2 *>(ct.fl + h0)[h];
                            const float2 fo = reinterpret_cast<const float2 *>(ct.fo + h0)[h];
                            l[h] = mul2(l[h], fl);
                            mv[h] = mul2(mv[h], fl);
                            if (TERMS == 2) left[h] = to_h2(h2_lo(left[h]) * fo.x, h2_hi(left[h]) * fo.y);
                        }
                        if (W)
                            for (int j = tid; j < kStep * i * kG; j += kWork) (&ct.w[0][0])[j] *= ct.fl[j % kG];
                        uint32_t o[kH];
#pragma unroll
                        for (int y = 0; y < SUBS; ++y) {
                            const int x = sub0 + y;          // columns of the leading terms, of the others
                            tmem_ld8_nowait(tmem + lanes + kColO + x * kG + h0, o);
                            tmem_wait_ld();
                            reg_fence(o);
#pragma unroll
                            for (int h = 0; h < kH; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * ct.fo[h0 + h]);
                            tmem_st8(tmem + lanes + kColO + x * kG + h0, o);
                        }
                        tmem_wait_st();
                    }
                    renew = 2;
                    continue;
                }
                // p = 2^y, and the weights p vs g in terms to shared memory: [tile][term][token][head]
                bool over = false;
                float faint = vs[0] < 0.0f ? 1.0f : vs[0];
                if (!HALF) faint = fminf(faint, vs[SUBS - 1] < 0.0f ? 1.0f : vs[SUBS - 1]);
                faint *= ct.least_g;
                if (__any_sync(kFull, faint < kFaint)) {   // p may grow where the weights do not
#pragma unroll
                    for (int h = 0; h < kH; ++h) over |= fmaxf(e[0][h], e[SUBS - 1][h]) > kMostY;
                }
                uint32_t high = 0u, rest[kH / 2];
#pragma unroll
                for (int h = 0; h < kH / 2; ++h) rest[h] = 0u;
#pragma unroll
                for (int sub = 0; sub < SUBS; ++sub) {
                    const float seen = vs[sub] < 0.0f ? 0.0f : vs[sub];   // no weight of -0: its sign would count as a high one
                    const f32x2 vs2 = pack2(seen, seen);
                    uint32_t word[2][TERMS];
#pragma unroll
                    for (int h = 0; h < kH; h += 4) {
                        float w[4];
                        uint32_t h2[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float &e0 = e[sub][h + 2 * j], &e1 = e[sub][h + 2 * j + 1];
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            const f32x2 w2 = mul2(mul2(pack2(e0, e1), vs2), reinterpret_cast<const f32x2 *>(ct.g + h0 + h)[j]);
                            unpack2(w2, w[2 * j], w[2 * j + 1]);
                            h2[j] = to_h2(w[2 * j], w[2 * j + 1]);
                        }
                        uint32_t r[2] = {rest[h / 2], rest[h / 2 + 1]};
                        split_weights<TERMS>(w, h2, word[h / 4], r);
                        rest[h / 2] = r[0];
                        rest[h / 2 + 1] = r[1];
                        high |= word[h / 4][0] + 0x08080808u;   // a leading term of 256 or more reaches bit 7
                    }
#pragma unroll
                    for (int y = 0; y < TERMS; ++y)
                        *reinterpret_cast<uint2 *>(sP + (t % L::kPBufs) * L::kStepP + (sub0 + sub) * L::kTileP +
                                                   y * L::kTermP + row * kG + h0) = make_uint2(word[0][y], word[1][y]);
                }
                over = renew == 0 && (over || (high & 0x80808080u) != 0u);
                fence_proxy_async();   // the weights are read by the tensor core
                tc_fence_before();
                if (!vote_barrier(over)) {
                    if (TERMS == 2)
#pragma unroll
                        for (int h = 0; h < kH / 2; ++h) left[h] = h2_add(left[h], rest[h]);
                    break;
                }
                renew = 1;
            }
#pragma unroll
            for (int sub = 0; sub < SUBS; ++sub) {
                const f32x2 vm2 = pack2(vm[sub], vm[sub]);
#pragma unroll
                for (int h = 0; h < kH / 2; ++h) {
                    const f32x2 e2 = pack2(e[sub][2 * h], e[sub][2 * h + 1]);
                    l[h] = add2(l[h], e2);
                    mv[h] = fma2(e2, vm2, mv[h]);
                }
            }
            if (W) {   // this block's sums: no other warp has this block and these columns
                float x[kH];
#pragma unroll
                for (int h = 0; h < kH; ++h) x[h] = HALF ? e[0][h] : e[0][h] + e[SUBS - 1][h];
                const float w = warp_sum8(x, lane);
                if ((lane & 3) == 0) ct.w[kStep * i + q][c0 + (lane >> 2)] = w;
            }
        }

        // ---- the unit's end: sums over the token lanes, outputs
        const int qi = u / a.n_kv_heads, g = u - qi * a.n_kv_heads;
        const size_t head0 = (size_t)qi * a.n_heads + (size_t)g * group;
        auto put = [&](int h, float x) {   // a warp's stores for one head are 32 neighbours
            const size_t at = (head0 + h) * kQDim + row;
            if (a.out_dt == QSA_F32) static_cast<float *>(a.out)[at] = x;
            else static_cast<uint16_t *>(a.out)[at] = (uint16_t)QFmt<F16>::bits_sat(x);   // values may pass the range, see store_row()
        };
        if (steps > 0) {
            float x[kH];
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                if (j == 2 && TERMS == 3) break;
#pragma unroll
                for (int h = 0; h < kH / 2; ++h) {
                    if (j < 2) {
                        unpack2(j ? mv[h] : l[h], x[2 * h], x[2 * h + 1]);
                    } else {
                        x[2 * h] = h2_lo(left[h]);
                        x[2 * h + 1] = h2_hi(left[h]);
                    }
                }
                const float sum = warp_sum8(x, lane);
                if ((lane & 3) == 0) ct.part[j][warp & 3][c0 + (lane >> 2)] = sum;
            }
            work_barrier();
            // o = (512 O ig + mean part ig + sum of p vm) / l: every warp makes all heads' factors for itself
            float *fin = ct.fin[warp][0];
            {
                const int h = lane & 15, w = lane >> 4;
                float tot[3];
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    tot[j] = 0.0f;
                    if (j == 2 && TERMS == 3) break;
                    tot[j] = ct.part[j][w][h] + ct.part[j][w + 2][h];
                    tot[j] += __shfl_xor_sync(kFull, tot[j], 16);
                    if (HALF) tot[j] += __shfl_xor_sync(kFull, tot[j], kH);   // both tiles' tokens
                }
                const float inv = 1.0f / tot[0], norm = split == 1 ? inv : 1.0f, ig = ct.ig[h];
                if (w == 0) {
                    fin[h] = ig;
                    fin[kG + h] = 512.0f * norm;
                    fin[3 * kG + h] = inv;
                    fin[2 * kG + h] = fmaf((7.5f / 16.0f) * tot[2], ig, tot[1]) * norm;
                    if (warp == 0) {
                        ct.sum[h] = tot[0];
                        if (split == 1 && a.lse && h < group) a.lse[head0 + h] = (log2f(tot[0]) - ct.nm[h]) * 0.6931471805599453f;
                    }
                }
                __syncwarp();
            }
            wait_all(&ct.obar, (uint32_t)(t - 1) & 1u, abort_flag);
            tc_fence_after();
            uint32_t o[2][kH];
#pragma unroll
            for (int j = 0; j < 2; ++j) tmem_ld8_nowait(tmem + lanes + kColO + j * kG + ho, o[j]);
            tmem_wait_ld();
            reg_fence(o[0]);
            reg_fence(o[1]);
            tc_fence_before();
            // this thread's dimension of its heads.  The codes' mean, 7.5, times what the rounding left of
            // the weights takes most of its effect away.
#pragma unroll
            for (int j = 0; j < kHO; j += 4) {
                const float4 ig = *reinterpret_cast<const float4 *>(fin + ho + j);
                const float4 up = *reinterpret_cast<const float4 *>(fin + kG + ho + j);
                const float4 add = *reinterpret_cast<const float4 *>(fin + 2 * kG + ho + j);
                const float igs[4] = {ig.x, ig.y, ig.z, ig.w}, ups[4] = {up.x, up.y, up.z, up.w};
                const float adds[4] = {add.x, add.y, add.z, add.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int h = ho + j + x;
                    const float sum = fmaf(__uint_as_float(o[1][j + x]), 0.0625f, __uint_as_float(o[0][j + x]));
                    const float y = fmaf(sum * ups[x], igs[x], adds[x]);
                    if (split > 1) reinterpret_cast<float *>(sK)[h * kQDim + row] = y;
                    else if (h < group) put(h, y);
                }
            }
            if (split == 1) {
                if (W && tid >= 64 && tid - 64 < nloc) {
                    const float4 *w4 = reinterpret_cast<const float4 *>(ct.w[tid - 64]);
                    const float4 *i4 = reinterpret_cast<const float4 *>(fin + 3 * kG);
                    float w = 0.0f;
#pragma unroll
                    for (int j = 0; j < kG / 4; ++j) {
                        const float4 x4 = w4[j], y4 = i4[j];
                        const int h = HALF ? 4 * j % kH : 4 * j;
                        w += h < group ? x4.x * y4.x : 0.0f;
                        w += h + 1 < group ? x4.y * y4.y : 0.0f;
                        w += h + 2 < group ? x4.z * y4.z : 0.0f;
                        w += h + 3 < group ? x4.w * y4.w : 0.0f;
                    }
                    a.weights[((size_t)qi * a.n_kv_heads + g) * a.k + un.slot[tid - 64]] = w;
                }
            }
        } else if (split == 1) {   // no visible token: o = 0
            for (int h = ho; h < min(group, ho + kHO); ++h) put(h, 0.0f);
            if (a.lse && tid < group) a.lse[head0 + tid] = -INFINITY;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.done[n & 1]);
    }
    }
    }
    __syncthreads();
    if (ct.abort) {   // a wait of some role gave up: what is in flight lands before any of the memory is used again
        if (warp >= kFetch) {      // each stage's last fill
            uint64_t *full = warp == kFetch ? ct.k_full : ct.v_full;
            for (int i = 0; i < 2; ++i)
                if (lap > 0 || i < stage) mbar_drain(&full[i], (i < stage ? lap : lap - 1u) & 1u);
        } else if (warp == kControl) {   // one more commit completes behind every product issued
            if (elect_one()) mma_commit(&ct.drained);
            __syncwarp();
            mbar_drain(&ct.drained, 0);
        }
        if (tid == 0 && a.flags) atomicOr(a.flags, QSA_FLAG_WAIT_TIMEOUT);
        __syncthreads();
    }
    if (warp == kControl) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(ct.tmem_base, kCols);
    }
    if (split > 1) {   // one unit per cluster
        // every CTA sends each head's partial output to the CTA that combines that head, and its (m, l)
        // to all; after the barrier each combines from its own memory
        const QUnit &un = ct.unit[0];
        const int qi = u0 / a.n_kv_heads, g = u0 - qi * a.n_kv_heads;
        const size_t head0 = (size_t)qi * a.n_heads + (size_t)g * group;
        const bool some = un.steps > 0;
        const int nh = kG / split;
        float *part = reinterpret_cast<float *>(sK);                 // this CTA's unnormalised output [16][128]
        float *recv = part + kG * kQDim;                             // [split][nh][128]
        cluster_sync();
        if (some)
            for (int x = tid; x < kG * 32; x += kThreads) {
                const int h = x >> 5, d4 = x & 31;
                st_cluster(reinterpret_cast<float4 *>(recv + (rank * nh + h % nh) * kQDim) + d4, h / nh,
                           reinterpret_cast<const float4 *>(part)[x]);
            }
        for (int x = tid; x < kG * split; x += kThreads) {
            const int h = x % kG;
            st_cluster(&ct.ml[rank][h], x / kG, make_float2(some ? -ct.nm[h] : -INFINITY, some ? ct.sum[h] : 0.0f));
        }
        cluster_sync();
        for (int x = tid; x < nh * kQDim; x += kThreads) {
            const int hh = x >> 7, d = x & 127, h = rank * nh + hh;
            float M = -INFINITY, Lsum = 0.0f, acc = 0.0f;
            for (int r = 0; r < split; ++r)
                if (ct.ml[r][h].y != 0.0f) M = fmaxf(M, ct.ml[r][h].x);
            for (int r = 0; r < split; ++r) {
                const float2 v = ct.ml[r][h];
                if (v.y != 0.0f) {   // a CTA without tokens took no part
                    const float f = exp2f(v.x - M);
                    Lsum = fmaf(f, v.y, Lsum);
                    acc = fmaf(f, recv[(r * nh + hh) * kQDim + d], acc);
                }
            }
            if (h < group) {
                const size_t at = (head0 + h) * kQDim + d;
                const float y = Lsum != 0.0f ? acc / Lsum : 0.0f;
                if (a.out_dt == QSA_F32) static_cast<float *>(a.out)[at] = y;
                else static_cast<uint16_t *>(a.out)[at] = (uint16_t)QFmt<F16>::bits_sat(y);
                if (a.lse && d == 0) a.lse[head0 + h] = Lsum != 0.0f ? (M + log2f(Lsum)) * 0.6931471805599453f : -INFINITY;
            }
        }
        if (W) {
            if (tid < kG) {   // this CTA's part of the total, per head
                float M = -INFINITY, Lsum = 0.0f;
                for (int r = 0; r < split; ++r)
                    if (ct.ml[r][tid].y != 0.0f) M = fmaxf(M, ct.ml[r][tid].x);
                for (int r = 0; r < split; ++r)
                    if (ct.ml[r][tid].y != 0.0f) Lsum = fmaf(exp2f(ct.ml[r][tid].x - M), ct.ml[r][tid].y, Lsum);
                ct.fl[tid] = some ? exp2f(-ct.nm[tid] - M) / Lsum : 0.0f;
            }
            __syncthreads();
            if (tid < un.nloc) {
                float w = 0.0f;
                for (int h = 0; h < group; ++h) w = fmaf(HALF ? ct.w[tid][h] + ct.w[tid][h + kH] : ct.w[tid][h], ct.fl[h], w);
                a.weights[((size_t)qi * a.n_kv_heads + g) * a.k + un.slot[un.b0 + tid]] = w;
            }
        }
    }
}

template <bool F16, bool W, bool HALF>
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
            st = check_cuda(cudaFuncSetAttribute(qattn_kernel<F16, W, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes),
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
    return check_cuda(cudaLaunchKernelEx(&cfg, qattn_kernel<F16, W, HALF>, p), "qattn_kernel launch");
}

}  // namespace

qsa_status launch_qcache_attention(const QAttnArgs &a, cudaStream_t s) {
    QParams p{};
    p.a = a;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    // few units: split each unit's steps over a cluster, doubling while every CTA has an SM of its own.  Split 1 /
    // 2 / 4 / 8 at k = 32, us: 4 units 11.8 / 10.6 / 8.6 / 8.0, 32 units 12.1 / 10.8 / 9.4 / 11.8, 76 units
    // 12.3 / 11.5 / 17.8 / 25.3, 152 units 12.6 / 15.6 / 27.6 / 43.6
    const long long units = (long long)a.nq * a.n_kv_heads;
    const int steps = (a.k + kStep - 1) / kStep;
    p.split = 1;
    while (p.split < kMaxSplit && p.split * 2 <= steps && units * p.split * 2 <= num_sms()) p.split *= 2;
    p.units = (int)units;
    const long long most = p.split > 1 ? units : 2ll * num_sms();
    const int grid = (int)(units < most ? units : most) * p.split;
    const bool half = a.n_heads / a.n_kv_heads <= kH;
    auto run = a.dt == QSA_F16 ? (a.weights ? (half ? launch_as<true, true, true> : launch_as<true, true, false>)
                                            : (half ? launch_as<true, false, true> : launch_as<true, false, false>))
                               : (a.weights ? (half ? launch_as<false, true, true> : launch_as<false, true, false>)
                                            : (half ? launch_as<false, false, true> : launch_as<false, false, false>));
    return run(p, grid, s);
}

}  // namespace qsa
