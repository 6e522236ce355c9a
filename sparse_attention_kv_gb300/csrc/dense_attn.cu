// dense_attn.cu -- attention of whole prompts over packed rows, and of drafted token trees over pages.
//
// The simplest form: a warp per (query, head).  32 keys at a time, a lane per key forms its logit; the softmax keeps a
// running maximum and sum; then a lane per four dimensions adds the keys' values up.  It reads K and V once per head.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.h"
#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int kWarps = 8;

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T, bool TREE>
__global__ void __launch_bounds__(32 * kWarps) dense_kernel(DenseArgs a) {
    __shared__ float qs[kWarps][128];
    wait_prior_grid();
    const int s = blockIdx.x, h = blockIdx.y, g = h / (a.n_heads / a.n_kv_heads);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    auto range = [&](const int32_t *cu, int most, int &c0, int &c1) {
        c0 = cu[s];
        c1 = cu[s + 1];
        if ((c0 < 0 || c1 < c0 || c1 > most) && threadIdx.x == 0) atomicOr(a.flags, QSA_FLAG_NBLOCKS_CLAMPED);
        c0 = min(max(c0, 0), most);
        c1 = min(max(c1, c0), most);
    };
    int q0, q1, k0 = 0, k1 = 0;
    range(a.cu_q, a.total_q, q0, q1);
    int past = 0;
    const int32_t *table = nullptr;
    if constexpr (TREE) {
        if (q1 - q0 > a.max_nodes) {
            q1 = q0 + a.max_nodes;
            if (threadIdx.x == 0) atomicOr(a.flags, QSA_FLAG_NBLOCKS_CLAMPED);
        }
        past = a.n_tokens[s];
        const int most = 64 * a.table.max_pages;
        if ((past < 0 || past > most) && threadIdx.x == 0) atomicOr(a.flags, QSA_FLAG_NBLOCKS_CLAMPED);
        past = min(max(past, 0), most);
        table = a.table.table + (size_t)s * a.table.stride;
    } else {
        range(a.cu_k, a.total_k, k0, k1);
    }
    const T *K = static_cast<const T *>(a.k.p) + g * a.k.head, *V = static_cast<const T *>(a.v.p) + g * a.v.head;
    const T *KC = static_cast<const T *>(a.kcache), *VC = static_cast<const T *>(a.vcache_t);
    for (int row = q0 + blockIdx.z * kWarps + wid; row < q1; row += gridDim.z * kWarps) {
        const int i = row - q0;
        unsigned long long sees = 0ull;
        int seen = 0;
        if constexpr (TREE) {
            for (int n = i; n >= 0;) {
                sees |= 1ull << n;
                int p = a.parents[q0 + n];
                if (p < -1 || p >= n) {
                    p = -1;
                    if (lane == 0) atomicOr(a.flags, QSA_FLAG_BAD_ID);
                }
                n = p;
            }
            seen = past + i + 1;
        } else {
            seen = max(0, (k1 - k0) - (q1 - q0) + i + 1);
        }
        const T *q = static_cast<const T *>(a.q.p) + (int64_t)row * a.q.token + (int64_t)h * a.q.head;
        __syncwarp();
        for (int d = lane; d < 128; d += 32) qs[wid][d] = to_f32(q[d]);
        __syncwarp();
        float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int t0 = 0; t0 < seen; t0 += 32) {
            const int t = t0 + lane;
            // where key t lies: row of K and V, or page and place
            bool ok = t < seen;
            int page = -1;
            if (TREE && ok) {
                if (t < past) {
                    page = table[t >> 6];
                    if (page < 0 || page >= a.table.n_pages) {
                        ok = false;
                        atomicOr(a.flags, QSA_FLAG_BAD_ID);
                    }
                } else {
                    ok = sees >> (t - past) & 1ull;
                }
            }
            float x = -INFINITY;
            if (ok) {
                const T *kr = page >= 0 ? KC + (((size_t)g * a.table.n_pages + page) * 64 + (t & 63)) * 128
                                        : K + (int64_t)(TREE ? q0 + t - past : k0 + t) * a.k.token;
                float dot = 0.0f;
                for (int d = 0; d < 128; ++d) dot += qs[wid][d] * to_f32(kr[d]);
                x = dot * a.scale;
            }
            float top = x;
            for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            const float m1 = fmaxf(m, top), ref = m1 == -INFINITY ? 0.0f : m1;
            const float turn = expf(m - ref), p = expf(x - ref);
            float sum = ok ? p : 0.0f;
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
            l = l * turn + sum;
            m = m1;
            for (int e = 0; e < 4; ++e) o[e] *= turn;
            for (int j = 0; j < 32 && t0 + j < seen; ++j) {
                const float w = __shfl_sync(~0u, p, j);
                const bool use = __shfl_sync(~0u, ok ? 1 : 0, j);
                const int pg = __shfl_sync(~0u, page, j), tj = t0 + j;
                if (!use) continue;
                for (int e = 0; e < 4; ++e) {
                    const int d = lane * 4 + e;
                    const T v = pg >= 0 ? VC[(((size_t)g * a.table.n_pages + pg) * 128 + d) * 64 + (tj & 63)]
                                        : V[(int64_t)(TREE ? q0 + tj - past : k0 + tj) * a.v.token + d];
                    o[e] += w * to_f32(v);
                }
            }
        }
        const size_t at = (size_t)row * a.n_heads + h;
        for (int e = 0; e < 4; ++e) {
            const float x = m == -INFINITY && l == 0.0f ? 0.0f : o[e] / l;
            const size_t to = at * 128 + lane * 4 + e;
            if (a.out_dt == QSA_F32) static_cast<float *>(a.out)[to] = x;
            else if (a.out_dt == QSA_BF16) static_cast<__nv_bfloat16 *>(a.out)[to] = __float2bfloat16(x);
            else static_cast<__half *>(a.out)[to] = __float2half(x);
        }
        if (lane == 0 && a.lse) a.lse[at] = l == 0.0f ? -INFINITY : m + logf(l);
    }
}

template <bool TREE>
qsa_status launch(const DenseArgs &a, cudaStream_t s) {
    const long long rows = TREE ? a.max_nodes : a.total_q;
    const dim3 grid((unsigned)a.n_seqs, (unsigned)a.n_heads, (unsigned)((rows + kWarps - 1) / kWarps < 64 ? (rows + kWarps - 1) / kWarps : 64));
    if (a.dt == QSA_BF16) dense_kernel<__nv_bfloat16, TREE><<<grid, 32 * kWarps, 0, s>>>(a);
    else dense_kernel<__half, TREE><<<grid, 32 * kWarps, 0, s>>>(a);
    return check_cuda(cudaGetLastError(), "dense_kernel launch");
}

}  // namespace

size_t attention_ws_bytes(int, int, int) { return 256; }
qsa_status launch_prompt_attention(const DenseArgs &a, cudaStream_t s) { return launch<false>(a, s); }
qsa_status launch_tree_attention(const DenseArgs &a, cudaStream_t s) { return launch<true>(a, s); }

}  // namespace qsa
