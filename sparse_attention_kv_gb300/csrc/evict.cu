// evict.cu -- eviction of KV blocks by accumulated attention weight: the selected
// blocks' weights added up per block, the blocks to keep, and the move of what is kept.
//
// 1. weights_add_kernel: acc[b] = decay * prev[b] + sum of the weights of the slots that
//    selected b.  Each CTA owns a range of blocks, reads every id, and adds the weights of
//    its own blocks in shared memory as 64-bit integers in units of 2^-36, so the result
//    does not depend on the order in which threads arrive.
// 2. evict_plan_kernel: one CTA per row finds the weight of the last block that stays by a
//    radix select over order-preserving keys (8 bits a pass), then emits the kept ids in
//    ascending order, ties to the lower id.
// 3. gather_blocks_kernel: one warp per (array, row, kept block) copies a block.
#include <climits>

#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr float kUnit = 68719476736.0f;   // 2^36
constexpr float kMaxWeight = QSA_MAX_BLOCK_WEIGHT;
constexpr int kAddThreads = 512;
constexpr int kAddBlocks = 512;           // blocks owned by a CTA

__global__ void __launch_bounds__(kAddThreads) weights_add_kernel(const float *__restrict__ weights,
                                                                  const int32_t *__restrict__ ids, int n_entries,
                                                                  int n_kv, int k, float decay, const float *prev,
                                                                  float *acc, int max_blocks, uint32_t *flags) {
    __shared__ unsigned long long sum[kAddBlocks];
    const int b0 = blockIdx.x * kAddBlocks;
    for (int i = threadIdx.x; i < kAddBlocks; i += kAddThreads) sum[i] = 0ull;
    __syncthreads();
    uint32_t bad = 0u;
    for (int e = threadIdx.x; e < n_entries; e += kAddThreads) {
        const int b = ids[e];
        if (blockIdx.x == 0 && b != -1 && (b < 0 || b >= max_blocks)) bad |= QSA_FLAG_BAD_ID;
        if (b < b0 || b >= b0 + kAddBlocks || b >= max_blocks) continue;
        const int q = e / k, j = e - q * k;
        const float *w = weights + (size_t)q * n_kv * k + j;
        unsigned long long add = 0ull;
        for (int g = 0; g < n_kv; ++g) {
            const float x = w[(size_t)g * k];
            if (!(x >= 0.0f && x <= kMaxWeight)) bad |= QSA_FLAG_BAD_WEIGHT;
            add += (unsigned long long)__float2ll_rn(fminf(fmaxf(x, 0.0f), kMaxWeight) * kUnit);   // NaN counts as 0
        }
        atomicAdd(&sum[b - b0], add);
    }
    if (bad && flags) atomicOr(flags, bad);
    __syncthreads();
    for (int i = threadIdx.x; i < kAddBlocks && b0 + i < max_blocks; i += kAddThreads) {
        // the sum in two halves, each exact in fp64 once scaled; fp32 once at the end
        const double s = (double)(sum[i] >> 32) * 0.0625 + (double)(uint32_t)sum[i] * (1.0 / 68719476736.0);
        const double p = prev ? (double)decay * (double)prev[b0 + i] : 0.0;
        acc[b0 + i] = (float)(p + s);
    }
}

constexpr int kPlanThreads = 1024;

// The order of eviction: weights as keys (NaN below every number), protected blocks above.
__device__ __forceinline__ uint32_t plan_key(float w, int b, int nb, int n_first, int n_last) {
    if (b < n_first || b >= nb - n_last) return 0xFFFFFFFFu;
    return w == w ? score_key(w) : 0u;
}

__global__ void __launch_bounds__(kPlanThreads) evict_plan_kernel(const float *__restrict__ weights, int64_t stride,
                                                                  const int32_t *__restrict__ n_tokens, int max_blocks,
                                                                  int n_keep, int n_first, int n_last, int32_t *keep,
                                                                  int32_t *new_tokens, uint32_t *flags) {
    __shared__ BlockScratch sm;
    const int row = blockIdx.x, tid = threadIdx.x;
    const float *w = weights + (size_t)row * stride;
    int32_t *out = keep + (size_t)row * n_keep;
    int nt = n_tokens[row];
    if (nt < 0 || (long long)nt > 64ll * max_blocks) {
        if (tid == 0 && flags) atomicOr(flags, QSA_FLAG_NBLOCKS_CLAMPED);
        nt = nt < 0 ? 0 : 64 * max_blocks;
    }
    const int nb = (int)(((long long)nt + 63) / 64);
    if (tid == 0) new_tokens[row] = nt - 64 * max(nb - n_keep, 0);
    if (nb <= n_keep) {
        for (int i = tid; i < n_keep; i += kPlanThreads) out[i] = i < nb ? i : -1;
        return;
    }
    // the n_keep-th largest key, 8 bits a pass
    uint32_t prefix = 0u, mask = 0u;
    int want = n_keep;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kPlanThreads) sm.hist[i] = 0u;
        __syncthreads();
        for (int b = tid; b < nb; b += kPlanThreads) {
            const uint32_t key = plan_key(w[b], b, nb, n_first, n_last);
            if ((key & mask) == prefix) atomicAdd(&sm.hist[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            int left = want, digit = 255;
            while (digit > 0 && (int)sm.hist[digit] < left) left -= (int)sm.hist[digit--];
            sm.misc[0] = digit;
            sm.misc[1] = left;
        }
        __syncthreads();
        prefix |= (uint32_t)sm.misc[0] << shift;
        mask |= 255u << shift;
        want = sm.misc[1];
        __syncthreads();
    }
    // ascending emit: keys above the threshold, and the first `want` equal to it
    int kept = 0, equal = 0;
    for (int b0 = 0; b0 < nb; b0 += kPlanThreads) {
        const int b = b0 + tid;
        const uint32_t key = b < nb ? plan_key(w[b], b, nb, n_first, n_last) : 0u;
        const bool eq = b < nb && key == prefix;
        int n_eq = 0;
        const int rank = equal + block_excl_scan<kPlanThreads>(eq ? 1 : 0, sm, n_eq);
        const bool take = b < nb && (key > prefix || (eq && rank < want));
        int n_take = 0;
        const int at = kept + block_excl_scan<kPlanThreads>(take ? 1 : 0, sm, n_take);
        if (take) out[at] = b;
        kept += n_take;
        equal += n_eq;
    }
}

constexpr int kGatherThreads = 256;
struct GatherParams {
    qsa_block_array a[QSA_GATHER_MAX_ARRAYS];
    long long first[QSA_GATHER_MAX_ARRAYS + 1];   // first warp of each array
    int n_arrays;
    int n_keep;
    const int32_t *keep;
    uint32_t *flags;
};

__global__ void __launch_bounds__(kGatherThreads) gather_blocks_kernel(const __grid_constant__ GatherParams p) {
    const int lane = threadIdx.x & 31;
    const long long n_warps = (long long)gridDim.x * (kGatherThreads / 32);
    for (long long w = (long long)blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5); w < p.first[p.n_arrays];
         w += n_warps) {
        int a = 0;
        while (w >= p.first[a + 1]) ++a;
        const qsa_block_array &x = p.a[a];
        const long long at = w - p.first[a];
        const int row = (int)(at / p.n_keep), i = (int)(at % p.n_keep);
        const int b = p.keep[i];
        if (b < 0 || b >= x.src_blocks) {
            if (b != -1 && lane == 0 && p.flags) atomicOr(p.flags, QSA_FLAG_BAD_ID);
            continue;
        }
        const uint8_t *src = static_cast<const uint8_t *>(x.src) + ((size_t)row * x.src_blocks + b) * x.block_bytes;
        uint8_t *dst = static_cast<uint8_t *>(x.dst) + ((size_t)row * x.dst_blocks + i) * x.block_bytes;
        if (((reinterpret_cast<uintptr_t>(x.src) | reinterpret_cast<uintptr_t>(x.dst) | (uintptr_t)x.block_bytes) & 15u) == 0u) {
            const int n = (int)(x.block_bytes >> 4);
#pragma unroll 4
            for (int j = lane; j < n; j += 32) reinterpret_cast<uint4 *>(dst)[j] = reinterpret_cast<const uint4 *>(src)[j];
        } else {
            const int n = (int)(x.block_bytes >> 2);
            for (int j = lane; j < n; j += 32)
                reinterpret_cast<uint32_t *>(dst)[j] = reinterpret_cast<const uint32_t *>(src)[j];
        }
    }
}

}  // namespace

qsa_status launch_weights_add(const WeightsAddArgs &a, cudaStream_t s) {
    const int grid = (a.max_blocks + kAddBlocks - 1) / kAddBlocks;
    weights_add_kernel<<<grid, kAddThreads, 0, s>>>(a.weights, a.ids, a.nq * a.k, a.n_kv_heads, a.k, a.decay, a.prev,
                                                    a.acc, a.max_blocks, a.flags);
    return check_cuda(cudaGetLastError(), "weights_add_kernel launch");
}

qsa_status launch_evict_plan(const EvictPlanArgs &a, cudaStream_t s) {
    evict_plan_kernel<<<a.n_rows, kPlanThreads, 0, s>>>(a.weights, a.stride, a.n_tokens, a.max_blocks, a.n_keep,
                                                        a.n_first, a.n_last, a.keep, a.new_tokens, a.flags);
    return check_cuda(cudaGetLastError(), "evict_plan_kernel launch");
}

qsa_status launch_gather_blocks(const qsa_block_array *arrays, int n_arrays, const int32_t *keep, int n_keep,
                                uint32_t *flags, cudaStream_t s) {
    GatherParams p{};
    p.n_arrays = n_arrays;
    p.n_keep = n_keep;
    p.keep = keep;
    p.flags = flags;
    for (int i = 0; i < n_arrays; ++i) {
        p.a[i] = arrays[i];
        p.first[i + 1] = p.first[i] + (long long)arrays[i].n_rows * n_keep;
    }
    const long long warps = p.first[n_arrays];
    const long long ctas = (warps + kGatherThreads / 32 - 1) / (kGatherThreads / 32);
    const long long most = 8ll * num_sms();
    gather_blocks_kernel<<<(unsigned)(ctas < most ? ctas : most), kGatherThreads, 0, s>>>(p);
    return check_cuda(cudaGetLastError(), "gather_blocks_kernel launch");
}

}  // namespace qsa
