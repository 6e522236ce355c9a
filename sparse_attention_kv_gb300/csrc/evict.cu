// evict.cu -- eviction of KV blocks by accumulated attention weight: the selected
// blocks' weights added up per block, the blocks to keep, and the move of what is kept.
//
// 1. acc[b] = decay * prev[b] + sum of the weights of the slots that selected b, added in shared
//    memory as 64-bit integers in units of 2^-36, so the result does not depend on the order in
//    which threads arrive.  Few entries: every CTA owns a range of blocks, reads all ids and takes its
//    own (weights_scan_kernel).  Many: the CTAs of one cluster share the blocks out, read an eighth
//    of the entries each and add to the owner's memory (weights_cluster_kernel).
// 2. evict_plan_kernel: one CTA per row holds the weights' order-preserving keys in registers, a
//    run of neighbouring blocks per thread, and finds the last key that stays bit by bit (a count
//    and a barrier each, 8.6 us at 8,125 blocks; two bits at a time took 13); one scan
//    then emits the kept ids in ascending order, ties to the lower id.  Rows past 16,384 blocks re-read their weights instead
//    (evict_plan_long_kernel, a radix select of 8 bits a pass).
// 3. gather_blocks_kernel: a warp copies 2 KB of a record, or as many small records as its lanes hold.
//
// Measured (warm graph): 1. 3.4 us for 3 queries x 4 KV heads x 32 slots over 4,032 blocks, 6.9 us for 256
// queries over 8,125 (every CTA reading all ids took 17.5); launches and one chain of loads.  2 and 3 together:
// 5.3 us to keep 128 of 257 blocks of one KV head; 55 us to keep 4,096 of 8,125 blocks of 4 (287 MB, of which
// the move takes 42 us, 6.9 TB/s: the copy rate).
#include <climits>
#include <mutex>

#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr float kUnit = 68719476736.0f;   // 2^36
constexpr float kMaxWeight = QSA_MAX_BLOCK_WEIGHT;
constexpr int kAddThreads = 512;
constexpr int kAddBlocks = 512;           // blocks owned by a CTA

// The integer sum of an entry's weights over the KV heads.
__device__ __forceinline__ unsigned long long entry_sum(const float *__restrict__ weights, int e, int n_kv, int k,
                                                        uint32_t &bad) {
    const int q = e / k, j = e - q * k;
    const float *w = weights + (size_t)q * n_kv * k + j;
    unsigned long long add = 0ull;
#pragma unroll 4
    for (int g = 0; g < n_kv; ++g) {
        const float x = w[(size_t)g * k];
        if (!(x >= 0.0f && x <= kMaxWeight)) bad |= QSA_FLAG_BAD_WEIGHT;
        add += (unsigned long long)__float2ll_rn(fminf(fmaxf(x, 0.0f), kMaxWeight) * kUnit);   // NaN counts as 0
    }
    return add;
}
// One block's result: the sum in two halves, each exact in fp64 once scaled; fp32 once at the end.
__device__ __forceinline__ float block_sum(unsigned long long sum, double decay, const float *prev, int b) {
    const double s = (double)(uint32_t)(sum >> 32) * 0.0625 + (double)(uint32_t)sum * (1.0 / 68719476736.0);
    return (float)((prev ? decay * (double)prev[b] : 0.0) + s);
}

__global__ void __launch_bounds__(kAddThreads) weights_scan_kernel(const float *__restrict__ weights,
                                                                   const int32_t *__restrict__ ids, int n_entries,
                                                                   int n_kv, int k, double decay, const float *prev,
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
        atomicAdd(&sum[b - b0], entry_sum(weights, e, n_kv, k, bad));
    }
    if (bad && flags) atomicOr(flags, bad);
    __syncthreads();
    for (int i = threadIdx.x; i < kAddBlocks && b0 + i < max_blocks; i += kAddThreads)
        acc[b0 + i] = block_sum(sum[i], decay, prev, b0 + i);
}

constexpr int kAddCluster = 8;
constexpr int kAddClusterThreads = 1024;
constexpr int kAddClusterBlocks = 28672;   // 8 bytes each in a CTA's shared memory

__global__ void __cluster_dims__(kAddCluster, 1, 1) __launch_bounds__(kAddClusterThreads)
    weights_cluster_kernel(const float *__restrict__ weights, const int32_t *__restrict__ ids, int n_entries, int n_kv,
                           int k, double decay, const float *prev, float *acc, int max_blocks, int per_cta,
                           uint32_t *flags) {
    extern __shared__ unsigned long long sums[];   // this CTA's blocks: blockIdx.x * per_cta ..
    for (int i = threadIdx.x; i < per_cta; i += kAddClusterThreads) sums[i] = 0ull;
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(sums));
    uint32_t bad = 0u;
    for (int e = blockIdx.x * kAddClusterThreads + threadIdx.x; e < n_entries; e += kAddCluster * kAddClusterThreads) {
        const int b = ids[e];
        if (b < 0 || b >= max_blocks) {
            if (b != -1) bad |= QSA_FLAG_BAD_ID;
            continue;
        }
        const unsigned long long add = entry_sum(weights, e, n_kv, k, bad);
        const int owner = b / per_cta;
        uint32_t at;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(base + (uint32_t)(b - owner * per_cta) * 8u), "r"(owner));
        asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(at), "l"(add) : "memory");
    }
    if (bad && flags) atomicOr(flags, bad);
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    const int b0 = blockIdx.x * per_cta;
    for (int i = threadIdx.x; i < per_cta && b0 + i < max_blocks; i += kAddClusterThreads)
        acc[b0 + i] = block_sum(sums[i], decay, prev, b0 + i);
}

constexpr int kPlanThreads = 1024;

// The order of eviction: weights as keys (NaN below every number), protected blocks above.
__device__ __forceinline__ uint32_t plan_key(float w, int b, int nb, int n_first, int n_last) {
    if (b < n_first || b >= nb - n_last) return 0xFFFFFFFFu;
    return w == w ? score_key(w) : 0u;
}

// What every plan kernel starts with: the row's tokens nt and its blocks; all of them kept: the answer at once.
// new_tokens may be n_tokens: every thread reads the old length before a barrier, and thread 0 stores the new one
// behind it (here, or at the kernel's end where fewer blocks are kept).
template <int NT>
__device__ __forceinline__ int plan_blocks(const int32_t *n_tokens, int row, int max_blocks, int n_keep, int32_t *out,
                                           int32_t *new_tokens, uint32_t *flags, int &nt) {
    nt = n_tokens[row];
    if (nt < 0 || (long long)nt > 64ll * max_blocks) {
        if (threadIdx.x == 0 && flags) atomicOr(flags, QSA_FLAG_NBLOCKS_CLAMPED);
        nt = nt < 0 ? 0 : 64 * max_blocks;
    }
    const int nb = (int)(((long long)nt + 63) / 64);
    if (nb <= n_keep) {
        __syncthreads();   // every thread takes this way: nb is the block's
        if (threadIdx.x == 0) new_tokens[row] = nt;
        for (int i = threadIdx.x; i < n_keep; i += NT) out[i] = i < nb ? i : -1;
    }
    return nb;
}

// E keys per thread, NT threads: rows of up to NT * E blocks.
template <int NT, int E>
__global__ void __launch_bounds__(NT) evict_plan_kernel(const float *__restrict__ weights, int64_t stride,
                                                        const int32_t *n_tokens, int max_blocks,
                                                        int n_keep, int n_first, int n_last, int32_t *keep,
                                                        int32_t *new_tokens, uint32_t *flags) {
    constexpr int NW = NT / 32;
    __shared__ int part[2][32];
    __shared__ BlockScratch sm;
    allow_dependent_launch();   // the move that follows may line up
    wait_prior_grid();
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float *w = weights + (size_t)row * stride;
    int32_t *out = keep + (size_t)row * n_keep;
    int nt;
    const int nb = plan_blocks<NT>(n_tokens, row, max_blocks, n_keep, out, new_tokens, flags, nt);
    if (nb <= n_keep) return;
    uint32_t key[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int b = tid * E + e;
        key[e] = b < nb ? plan_key(w[b], b, nb, n_first, n_last) : 0u;
    }
    // the largest T with at least n_keep keys >= T, bit by bit, until a count meets n_keep.  Keys past the row are
    // 0: a T above 0 does not count them, and T stays 0 only when fewer than n_keep keys are above 0.
    uint32_t T = 0u;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t M = T | (1u << bit);
        int mine = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) mine += key[e] >= M ? 1 : 0;
        mine = __reduce_add_sync(kFull, mine);
        int *p = part[bit & 1];
        if (lane == 0) p[warp] = mine;
        __syncthreads();
        const int all = __reduce_add_sync(kFull, lane < NW ? p[lane] : 0);
        if (all >= n_keep) T = M;
        if (all == n_keep) {   // exactly these: the keys above M - 1
            T = M - 1u;
            break;
        }
    }
    // ascending emit: keys above T, and the first of those equal to it
    int above = 0, equal = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const bool in = tid * E + e < nb;
        above += in && key[e] > T ? 1 : 0;
        equal += in && key[e] == T ? 1 : 0;
    }
    if (tid == 0) new_tokens[row] = nt - 64 * (nb - n_keep);   // barriers lie behind: every thread has read n_tokens
    int total = 0;   // both counts in one scan: rows have at most 2^14 blocks
    const uint32_t before = (uint32_t)block_excl_scan<NT>(above | (equal << 16), sm, total);
    const int want = n_keep - (total & 0xFFFF);
    int at = (int)(before & 0xFFFFu), eq = (int)(before >> 16);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int b = tid * E + e;
        if (b >= nb) continue;
        if (key[e] > T) out[min(eq, want) + at++] = b;
        if (key[e] == T) {
            if (eq < want) out[eq + at] = b;
            ++eq;
        }
    }
}

__global__ void __launch_bounds__(kPlanThreads) evict_plan_long_kernel(const float *__restrict__ weights, int64_t stride,
                                                                  const int32_t *n_tokens, int max_blocks,
                                                                  int n_keep, int n_first, int n_last, int32_t *keep,
                                                                  int32_t *new_tokens, uint32_t *flags) {
    __shared__ BlockScratch sm;
    wait_prior_grid();
    const int row = blockIdx.x, tid = threadIdx.x;
    const float *w = weights + (size_t)row * stride;
    int32_t *out = keep + (size_t)row * n_keep;
    int nt;
    const int nb = plan_blocks<kPlanThreads>(n_tokens, row, max_blocks, n_keep, out, new_tokens, flags, nt);
    if (nb <= n_keep) return;
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
    if (tid == 0) new_tokens[row] = nt - 64 * (nb - n_keep);   // barriers lie behind: every thread has read n_tokens
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
constexpr int kBatch = 4;   // 16-byte (or 4-byte) units per lane in flight
// How an array's records are dealt to warps: `lanes` lanes per record (a power of two) and so 32 / lanes records
// per warp, or, for records of more than 32 units, `pieces` warps per record.
struct GatherArray {
    const uint8_t *src;
    uint8_t *dst;
    uint32_t units;          // per record, of 16 bytes (wide) or 4
    int wide;
    int lanes, pieces;
    uint32_t groups;         // per row: groups of 32 / lanes records
    int src_blocks, dst_blocks;
};
struct GatherParams {
    GatherArray a[QSA_GATHER_MAX_ARRAYS];
    long long first[QSA_GATHER_MAX_ARRAYS + 1];   // first warp of each array
    int n_arrays;
    int n_keep;
    const int32_t *keep;
    uint32_t *flags;
};

template <typename T>
__device__ __forceinline__ void copy_units(const uint8_t *src, uint8_t *dst, uint32_t at, uint32_t end, uint32_t step) {
    const T *s = reinterpret_cast<const T *>(src);
    T *d = reinterpret_cast<T *>(dst);
    T x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
        if (at + i * step < end) x[i] = __ldcs(s + at + i * step);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
        if (at + i * step < end) __stcs(d + at + i * step, x[i]);
}

__global__ void __launch_bounds__(kGatherThreads) gather_blocks_kernel(const __grid_constant__ GatherParams p) {
    const int lane = threadIdx.x & 31;
    const long long n_warps = (long long)gridDim.x * (kGatherThreads / 32), all = p.first[p.n_arrays];
    wait_prior_grid();
    for (long long w = (long long)blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5); w < all; w += n_warps) {
        int a = 0;
        while (w >= p.first[a + 1]) ++a;
        const GatherArray &x = p.a[a];
        const uint64_t at = (uint64_t)(w - p.first[a]);
        const uint32_t group = (uint32_t)(at / (uint32_t)x.pieces), piece = (uint32_t)(at - (uint64_t)group * x.pieces);
        const uint32_t row = group / x.groups;
        const uint32_t i = (group - row * x.groups) * (32u / x.lanes) + lane / x.lanes;
        if (i >= (uint32_t)p.n_keep) continue;
        const int b = p.keep[i];
        if (b < 0 || b >= x.src_blocks) {
            if (b != -1 && lane % x.lanes == 0 && p.flags) atomicOr(p.flags, QSA_FLAG_BAD_ID);
            continue;
        }
        const size_t bytes = (size_t)x.units * (x.wide ? 16 : 4);
        const uint8_t *src = x.src + ((size_t)row * x.src_blocks + b) * bytes;
        uint8_t *dst = x.dst + ((size_t)row * x.dst_blocks + i) * bytes;
        const uint32_t from = piece * (32u * kBatch) + lane % x.lanes;
        if (x.wide) copy_units<uint4>(src, dst, from, x.units, (uint32_t)x.lanes);
        else copy_units<uint32_t>(src, dst, from, x.units, (uint32_t)x.lanes);
    }
}

}  // namespace

// Launch as a programmatic dependent of the work before it on the stream: the kernel waits for it at entry.
template <typename... Params, typename... Args>
static qsa_status launch_dependent(const char *what, void (*kern)(Params...), int grid, int threads, size_t smem,
                                   cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...), what);
}

// Up to this many entries every CTA scans them all, two per thread.  Scan / cluster, us, 8,125 blocks: 3.7 / 4.9 at
// 256 entries, 5.0 / 6.1 at 1,024, 6.8 / 6.1 at 2,048, 17.5 / 6.6 at 8,192; 2,048 blocks: 3.6 / 3.6, 4.8 / 4.4,
// 7.1 / 4.9, 18.4 / 5.5.
constexpr int kScanEntries = 1024;

qsa_status launch_weights_add(const WeightsAddArgs &a, cudaStream_t s) {
    const int entries = a.nq * a.k;
    const int per_cta = (a.max_blocks + kAddCluster - 1) / kAddCluster;
    if (entries > kScanEntries && per_cta <= kAddClusterBlocks) {
        static std::mutex mu;
        static bool opted_in[64] = {false};
        int dev = 0;
        qsa_status st = check_cuda(cudaGetDevice(&dev), "cudaGetDevice");
        if (st != QSA_OK) return st;
        if (dev < 0 || dev >= 64) return fail(QSA_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
        {
            std::lock_guard<std::mutex> lock(mu);
            if (!opted_in[dev]) {
                st = check_cuda(cudaFuncSetAttribute(weights_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     kAddClusterBlocks * 8),
                                "cudaFuncSetAttribute(block weights)");
                if (st != QSA_OK) return st;
                opted_in[dev] = true;
            }
        }
        weights_cluster_kernel<<<kAddCluster, kAddClusterThreads, (size_t)per_cta * 8, s>>>(
            a.weights, a.ids, entries, a.n_kv_heads, a.k, a.decay, a.prev, a.acc, a.max_blocks, per_cta, a.flags);
        return check_cuda(cudaGetLastError(), "weights_cluster_kernel launch");
    }
    const int grid = (a.max_blocks + kAddBlocks - 1) / kAddBlocks;
    weights_scan_kernel<<<grid, kAddThreads, 0, s>>>(a.weights, a.ids, entries, a.n_kv_heads, a.k, a.decay, a.prev, a.acc,
                                                     a.max_blocks, a.flags);
    return check_cuda(cudaGetLastError(), "weights_scan_kernel launch");
}

qsa_status launch_evict_plan(const EvictPlanArgs &a, cudaStream_t s) {
    auto run = [&](auto *kern, int threads) {
        return launch_dependent("evict_plan_kernel launch", kern, a.n_rows, threads, 0, s, a.weights, a.stride, a.n_tokens,
                                a.max_blocks, a.n_keep, a.n_first, a.n_last, a.keep, a.new_tokens, a.flags);
    };
    // Few keys per thread and few warps: a step's barrier is cheaper among fewer, its compares among more.  us with
    // 256 / 512 / 1,024 threads: 257 blocks 3.6 / 4.1 / 5.3, 1,000 blocks 3.6 / 4.0 / 5.0, 2,048 blocks 4.4 / 4.0 / 5.0,
    // 4,000 blocks 7.2 / 6.1 / 6.0, 8,125 blocks 13.5 / 9.9 / 8.6
    if (a.max_blocks <= 1024) return run(evict_plan_kernel<256, 4>, 256);
    if (a.max_blocks <= 2048) return run(evict_plan_kernel<512, 4>, 512);
    if (a.max_blocks <= 4096) return run(evict_plan_kernel<512, 8>, 512);
    if (a.max_blocks <= 8192) return run(evict_plan_kernel<1024, 8>, 1024);
    if (a.max_blocks <= 16384) return run(evict_plan_kernel<1024, 16>, 1024);
    return run(evict_plan_long_kernel, kPlanThreads);
}

qsa_status launch_gather_blocks(const qsa_block_array *arrays, int n_arrays, const int32_t *keep, int n_keep,
                                uint32_t *flags, cudaStream_t s) {
    GatherParams p{};
    p.n_arrays = n_arrays;
    p.n_keep = n_keep;
    p.keep = keep;
    p.flags = flags;
    for (int i = 0; i < n_arrays; ++i) {
        const qsa_block_array &x = arrays[i];
        GatherArray &y = p.a[i];
        y.src = static_cast<const uint8_t *>(x.src);
        y.dst = static_cast<uint8_t *>(x.dst);
        y.wide = ((reinterpret_cast<uintptr_t>(x.src) | reinterpret_cast<uintptr_t>(x.dst) | (uintptr_t)x.block_bytes) & 15u) == 0u;
        y.units = (uint32_t)(x.block_bytes >> (y.wide ? 4 : 2));
        y.lanes = 1;
        while (y.lanes < 32 && (uint32_t)y.lanes < y.units) y.lanes *= 2;
        y.pieces = (int)((y.units + 32u * kBatch - 1) / (32u * kBatch));
        y.groups = (uint32_t)((n_keep + 32 / y.lanes - 1) / (32 / y.lanes));
        y.src_blocks = x.src_blocks;
        y.dst_blocks = x.dst_blocks;
        p.first[i + 1] = p.first[i] + (long long)x.n_rows * y.groups * y.pieces;
    }
    const long long warps = p.first[n_arrays];
    const long long ctas = (warps + kGatherThreads / 32 - 1) / (kGatherThreads / 32);
    const long long most = 8ll * num_sms();
    return launch_dependent("gather_blocks_kernel launch", gather_blocks_kernel, (int)(ctas < most ? ctas : most),
                            kGatherThreads, 0, s, p);
}

}  // namespace qsa
