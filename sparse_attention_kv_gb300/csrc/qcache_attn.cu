// qcache_attn.cu -- selection attention over the 4-bit KV cache.
//
//   s_t = scale * dot(q[h], K[t]),  o[h] = sum_t p_t V[t] / sum_t p_t,  p_t = exp(s_t - m),
//   weight[slot] = sum over the group's heads and the slot's tokens of p_t / sum p
//
// over the tokens of the distinct selected blocks below n_tokens, K[t] and V[t] the
// 4-bit rows' values scale * code + minimum.  One CTA (128 threads) per (query, KV
// head), one block at a time: dequantised K rows against all heads, a running maximum
// and sum per head, then P.V with one head dimension per thread.
#include <cmath>

#include "qcache.cuh"
#include "qsa_device.cuh"

namespace qsa {
namespace {

constexpr int kG = 16;   // most query heads per KV head
constexpr int kSel = QSA_ATTN_MAX_K;

struct QAttnSmem {
    float q[kG][kQDim];
    float s[kG][kQBlockTok];
    float vs[kQBlockTok], vm[kQBlockTok];
    float m[kG], l[kG], f[kG];
    float w[kSel][kG];    // a slot's sum of exp(s - m) at the running maximum
    int32_t id[kSel];     // the block of a slot, -1: none, out of context or a repeat
};

template <bool F16>
__global__ void __launch_bounds__(128) qattn_kernel(const QAttnArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    QAttnSmem &sm = *reinterpret_cast<QAttnSmem *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int qi = blockIdx.x / a.n_kv_heads, g = blockIdx.x % a.n_kv_heads;
    const int group = a.n_heads / a.n_kv_heads, nb_cap = a.capacity / kQBlockTok;
    int ntok = a.n_tokens[qi];
    if (ntok < 0 || ntok > a.capacity) {
        if (tid == 0 && g == 0 && a.flags) atomicOr(a.flags, QSA_FLAG_NBLOCKS_CLAMPED);
        ntok = ntok < 0 ? 0 : a.capacity;
    }
    const int nb = (ntok + kQBlockTok - 1) / kQBlockTok;
    const int32_t *ids = a.ids + (size_t)qi * a.k;
    if (tid < a.k) {
        const int32_t b = ids[tid];
        bool take = b >= 0 && b < nb;
        if (!take && b != -1 && a.flags) atomicOr(a.flags, QSA_FLAG_BAD_ID);
        for (int i = 0; take && i < tid; ++i) take = ids[i] != b;
        sm.id[tid] = take ? b : -1;
    }
    const uint16_t *qrow = static_cast<const uint16_t *>(a.qa) + qi * a.q_stride + (size_t)(g * group) * a.q_head_stride;
    for (int h = 0; h < kG; ++h) {
        const uint32_t x = h < group ? qrow[h * a.q_head_stride + tid] : 0u;
        sm.q[h][tid] = QFmt<F16>::lo(x);
    }
    if (tid < kG) {
        sm.m[tid] = -INFINITY;
        sm.l[tid] = 0.0f;
    }
    for (int i = tid; i < kSel * kG; i += 128) sm.w[i / kG][i % kG] = 0.0f;
    float acc[kG];
#pragma unroll
    for (int h = 0; h < kG; ++h) acc[h] = 0.0f;
    __syncthreads();
    for (int j = 0; j < a.k; ++j) {
        const int b = sm.id[j];
        if (b < 0) continue;
        const uint8_t *rec = static_cast<const uint8_t *>(a.cache) + qrec_offset(g, nb_cap, b);
        const int nt = min(kQBlockTok, ntok - b * kQBlockTok);
        {   // logits: token tid & 63, half of the heads
            const int t = tid & 63, h0 = (tid >> 6) * 8;
            const uint32_t pair = *reinterpret_cast<const uint32_t *>(rec + kQOffKPair + t * 4);
            const float ks = QFmt<F16>::lo(pair), km = QFmt<F16>::hi(pair);
            float s[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) s[h] = 0.0f;
            for (int c = 0; c < 4; ++c)
                for (int i = 0; i < 16; ++i) {
                    const uint32_t x = rec[c * 1024 + t * 16 + i];
                    const float lo = fmaf(ks, (float)(x & 15u), km), hi = fmaf(ks, (float)(x >> 4), km);
#pragma unroll
                    for (int h = 0; h < 8; ++h)
                        s[h] = fmaf(lo, sm.q[h0 + h][16 * c + i], fmaf(hi, sm.q[h0 + h][64 + 16 * c + i], s[h]));
                }
#pragma unroll
            for (int h = 0; h < 8; ++h) sm.s[h0 + h][t] = t < nt ? s[h] * a.scale : -INFINITY;
            if (tid < 64) {
                const uint32_t vp = *reinterpret_cast<const uint32_t *>(rec + kQOffVPair + t * 4);
                sm.vs[t] = t < nt ? QFmt<F16>::lo(vp) : 0.0f;
                sm.vm[t] = t < nt ? QFmt<F16>::hi(vp) : 0.0f;
            }
        }
        __syncthreads();
        for (int h = warp; h < kG; h += 4) {   // running maximum and sum, one warp per head
            const float s0 = sm.s[h][lane], s1 = sm.s[h][lane + 32];
            float mx = fmaxf(s0, s1);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
            const float m0 = sm.m[h], m1 = fmaxf(m0, mx);
            const float e0 = expf(s0 - m1), e1 = expf(s1 - m1);
            sm.s[h][lane] = e0;
            sm.s[h][lane + 32] = e1;
            float sum = e0 + e1;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            const float f = expf(m0 - m1);
            for (int i = lane; i < j; i += 32) sm.w[i][h] *= f;
            __syncwarp();
            if (lane == 0) {
                sm.f[h] = f;
                sm.m[h] = m1;
                sm.l[h] = sm.l[h] * f + sum;
                sm.w[j][h] = sum;
            }
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kG; ++h) acc[h] *= sm.f[h];
        for (int t = 0; t < nt; ++t) {   // dimension tid
            const uint32_t x = rec[kQOffV + ((t & 31) >> 4) * 2048 + tid * 16 + (t & 15)];
            const float v = fmaf(sm.vs[t], (float)(t < 32 ? x & 15u : x >> 4), sm.vm[t]);
#pragma unroll
            for (int h = 0; h < kG; ++h) acc[h] = fmaf(sm.s[h][t], v, acc[h]);
        }
        __syncthreads();
    }
    for (int h = 0; h < group; ++h) {
        const size_t head = (size_t)qi * a.n_heads + g * group + h;
        const float l = sm.l[h], o = l != 0.0f ? acc[h] / l : 0.0f;
        if (a.out_dt == QSA_F32) static_cast<float *>(a.out)[head * kQDim + tid] = o;
        else static_cast<uint16_t *>(a.out)[head * kQDim + tid] = (uint16_t)QFmt<F16>::bits(o);
        if (a.lse && tid == 0) a.lse[head] = l != 0.0f ? sm.m[h] + logf(l) : -INFINITY;
    }
    if (a.weights && tid < a.k) {
        float w = 0.0f;
        for (int h = 0; h < group; ++h) w += sm.l[h] != 0.0f ? sm.w[tid][h] / sm.l[h] : 0.0f;
        a.weights[((size_t)qi * a.n_kv_heads + g) * a.k + tid] = w;
    }
}

}  // namespace

qsa_status launch_qcache_attention(const QAttnArgs &a, cudaStream_t s) {
    auto *kern = a.dt == QSA_F16 ? qattn_kernel<true> : qattn_kernel<false>;
    kern<<<a.nq * a.n_kv_heads, 128, sizeof(QAttnSmem), s>>>(a);
    return check_cuda(cudaGetLastError(), "qattn_kernel launch");
}

}  // namespace qsa
