// qcache_api.cu -- the C ABI of the 4-bit KV cache and of the eviction: argument checks.
#include <cfloat>

#include "qsa_internal.h"

namespace qsa {
namespace {

bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1u)) != 0; }

qsa_status check_flags_ws(const void *ws, size_t ws_bytes) {
    if (ws && (ws_bytes < 256 || misaligned(ws, 256)))
        return fail(QSA_ERR_WORKSPACE, "workspace must be 256-byte aligned and hold at least 256 bytes");
    return QSA_OK;
}

qsa_status check_cache(int n_kv_heads, int head_dim, int capacity, qsa_dtype dt) {
    if (head_dim != QSA_HEAD_DIM)
        return fail(QSA_ERR_INVALID_ARG, "head_dim must be %d (got %d)", QSA_HEAD_DIM, head_dim);
    if (n_kv_heads < 1 || n_kv_heads > 65535)   // one grid row per KV head
        return fail(QSA_ERR_INVALID_ARG, "n_kv_heads must be in [1, 65535] (got %d)", n_kv_heads);
    if (capacity < 64 || capacity % 64 || capacity / 64 > QSA_MAX_BLOCKS)
        return fail(QSA_ERR_INVALID_ARG, "capacity must be a positive multiple of 64 of at most %d blocks (got %d)",
                    QSA_MAX_BLOCKS, capacity);
    if (dt != QSA_BF16 && dt != QSA_F16)
        return fail(QSA_ERR_UNSUPPORTED, "the 4-bit cache takes bf16 or fp16 rows (dtype %d)", (int)dt);
    return QSA_OK;
}

qsa_status check_strides(int64_t a, int64_t b, const char *what) {
    if (a % 8 || b % 8)
        return fail(QSA_ERR_INVALID_ARG, "%s strides must be multiples of 8 elements (got %lld, %lld)", what,
                    (long long)a, (long long)b);
    return QSA_OK;
}

qsa_status check_rows(const void *k, int64_t kt, int64_t kh, const void *v, int64_t vt, int64_t vh, const void *cache,
                      int n, int n_kv_heads, int head_dim, int capacity, qsa_dtype dt) {
    if (!k || !v || !cache) return fail(QSA_ERR_INVALID_ARG, "NULL k, v or cache");
    qsa_status st = check_cache(n_kv_heads, head_dim, capacity, dt);
    if (st != QSA_OK) return st;
    if ((st = check_strides(kt, kh, "k")) != QSA_OK || (st = check_strides(vt, vh, "v")) != QSA_OK) return st;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(cache, 16))
        return fail(QSA_ERR_INVALID_ARG, "k, v and cache must be 16-byte aligned");
    if (n < 0 || n > capacity) return fail(QSA_ERR_INVALID_ARG, "n must be in [0, capacity] (got %d)", n);
    return QSA_OK;
}

// Whether [a, a + an) and [b, b + bn) share a byte.
bool overlap(const void *a, size_t an, const void *b, size_t bn) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bn && b0 < a0 + an;
}

uint32_t *flags_of(void *ws) { return static_cast<uint32_t *>(ws); }

}  // namespace
}  // namespace qsa

using namespace qsa;

extern "C" {

size_t qsa_qcache_bytes(int n_kv_heads, int capacity) {
    if (n_kv_heads < 1 || n_kv_heads > 65535 || capacity < 64 || capacity % 64 || capacity / 64 > QSA_MAX_BLOCKS) return 0;
    return (size_t)n_kv_heads * (size_t)(capacity / 64) * QSA_QCACHE_BLOCK_BYTES;
}

qsa_status qsa_qcache_append(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                             int64_t v_token_stride, int64_t v_head_stride, qsa_dtype dt, int n, int n_kv_heads,
                             int head_dim, int first, const int32_t *first_dev, void *cache, int capacity, void *ws,
                             size_t ws_bytes, qsa_stream stream) {
    qsa_status st = check_rows(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, cache, n, n_kv_heads,
                               head_dim, capacity, dt);
    if (st != QSA_OK) return st;
    if (!first_dev && (first < 0 || (long long)first + n > capacity))
        return fail(QSA_ERR_INVALID_ARG, "positions [%d, %d + %d) outside [0, %d)", first, first, n, capacity);
    if ((st = check_flags_ws(ws, ws_bytes)) != QSA_OK) return st;
    if (n == 0) return QSA_OK;
    QAppendArgs a{};
    a.k = k;
    a.v = v;
    a.k_token_stride = k_token_stride;
    a.k_head_stride = k_head_stride;
    a.v_token_stride = v_token_stride;
    a.v_head_stride = v_head_stride;
    a.dt = dt;
    a.n = n;
    a.n_kv_heads = n_kv_heads;
    a.first = first;
    a.first_dev = first_dev;
    a.cache = cache;
    a.capacity = capacity;
    a.flags = flags_of(ws);
    return launch_qcache_append(a, static_cast<cudaStream_t>(stream));
}

qsa_status qsa_qcache_load(const void *cache, qsa_dtype dt, int n_kv_heads, int head_dim, int capacity, int first,
                           int n, void *k, int64_t k_token_stride, int64_t k_head_stride, void *v,
                           int64_t v_token_stride, int64_t v_head_stride, qsa_stream stream) {
    qsa_status st = check_rows(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, cache, n, n_kv_heads,
                               head_dim, capacity, dt);
    if (st != QSA_OK) return st;
    if (first < 0 || (long long)first + n > capacity)
        return fail(QSA_ERR_INVALID_ARG, "positions [%d, %d + %d) outside [0, %d)", first, first, n, capacity);
    if (n == 0) return QSA_OK;
    QLoadArgs a{};
    a.cache = cache;
    a.dt = dt;
    a.n_kv_heads = n_kv_heads;
    a.capacity = capacity;
    a.first = first;
    a.n = n;
    a.k = k;
    a.v = v;
    a.k_token_stride = k_token_stride;
    a.k_head_stride = k_head_stride;
    a.v_token_stride = v_token_stride;
    a.v_head_stride = v_head_stride;
    return launch_qcache_load(a, static_cast<cudaStream_t>(stream));
}

qsa_status qsa_select_attention_qcache(const void *qa, int64_t q_stride, int64_t q_head_stride, qsa_dtype dt,
                                       const void *cache, const int32_t *ids, int k, const int32_t *n_tokens, int nq,
                                       int n_heads, int n_kv_heads, int head_dim, int capacity, float scale, void *out,
                                       qsa_dtype out_dt, float *lse, float *weights, void *ws, size_t ws_bytes,
                                       qsa_stream stream) {
    if (!qa || !cache || !ids || !n_tokens || !out)
        return fail(QSA_ERR_INVALID_ARG, "NULL qa, cache, ids, n_tokens or out");
    if (nq < 1) return fail(QSA_ERR_INVALID_ARG, "nq must be >= 1 (got %d)", nq);
    qsa_status st = check_cache(n_kv_heads, head_dim, capacity, dt);
    if (st != QSA_OK) return st;
    if (n_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > QSA_ATTN_GROUP)
        return fail(QSA_ERR_INVALID_ARG, "n_heads must be 1 to %d times n_kv_heads (got %d heads, %d KV heads)",
                    QSA_ATTN_GROUP, n_heads, n_kv_heads);
    if (k < 1 || k > QSA_ATTN_MAX_K)
        return fail(QSA_ERR_INVALID_ARG, "k must be in [1, %d] (got %d)", QSA_ATTN_MAX_K, k);
    if ((long long)nq * n_kv_heads >= (1ll << 28)) return fail(QSA_ERR_INVALID_ARG, "nq * n_kv_heads too large");
    if ((st = check_strides(q_stride, q_head_stride, "qa")) != QSA_OK) return st;
    if (misaligned(qa, 16) || misaligned(cache, 16) || misaligned(out, 16))
        return fail(QSA_ERR_INVALID_ARG, "qa, cache and out must be 16-byte aligned");
    if (!(scale > 0.0f) || !(scale <= 3.4e38f)) return fail(QSA_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (out_dt != QSA_F32 && out_dt != dt)
        return fail(QSA_ERR_INVALID_ARG, "out must be fp32 or of the inputs' dtype (got %d)", (int)out_dt);
    if ((st = check_flags_ws(ws, ws_bytes)) != QSA_OK) return st;
    QAttnArgs a{};
    a.qa = qa;
    a.q_stride = q_stride;
    a.q_head_stride = q_head_stride;
    a.dt = dt;
    a.cache = cache;
    a.ids = ids;
    a.k = k;
    a.n_tokens = n_tokens;
    a.nq = nq;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.capacity = capacity;
    a.scale = scale;
    a.out = out;
    a.out_dt = out_dt;
    a.lse = lse;
    a.weights = weights;
    a.flags = flags_of(ws);
    return launch_qcache_attention(a, static_cast<cudaStream_t>(stream));
}

qsa_status qsa_block_weights_add(const float *weights, const int32_t *ids, int nq, int n_kv_heads, int k, double decay,
                                 const float *prev, float *acc, int max_blocks, void *ws, size_t ws_bytes,
                                 qsa_stream stream) {
    if (!weights || !ids || !acc) return fail(QSA_ERR_INVALID_ARG, "NULL weights, ids or acc");
    if (nq < 1 || n_kv_heads < 1 || k < 1)
        return fail(QSA_ERR_INVALID_ARG, "nq, n_kv_heads and k must be >= 1 (got %d, %d, %d)", nq, n_kv_heads, k);
    // the largest sum, 2^22 weights of 2^5 in units of 2^-36, is below 2^64
    if ((long long)nq * n_kv_heads > (1ll << 22) || (long long)nq * n_kv_heads * k > (1ll << 22))
        return fail(QSA_ERR_INVALID_ARG, "nq * n_kv_heads * k too large (at most %d)", 1 << 22);
    if (max_blocks < 1 || max_blocks > QSA_MAX_BLOCKS)
        return fail(QSA_ERR_INVALID_ARG, "max_blocks must be in [1, %d] (got %d)", QSA_MAX_BLOCKS, max_blocks);
    if (!(decay >= 0.0) || !(decay <= DBL_MAX)) return fail(QSA_ERR_INVALID_ARG, "decay must be finite and >= 0");
    const size_t acc_bytes = (size_t)max_blocks * sizeof(float), entries = (size_t)nq * k;
    if (prev && prev != acc && overlap(acc, acc_bytes, prev, acc_bytes))
        return fail(QSA_ERR_INVALID_ARG, "prev must be acc itself or not overlap it");
    qsa_status st = check_flags_ws(ws, ws_bytes);
    if (st != QSA_OK) return st;
    if (overlap(acc, acc_bytes, weights, entries * n_kv_heads * sizeof(float)) ||
        overlap(acc, acc_bytes, ids, entries * sizeof(int32_t)))
        return fail(QSA_ERR_INVALID_ARG, "acc must not overlap weights or ids");
    WeightsAddArgs a{};
    a.weights = weights;
    a.ids = ids;
    a.nq = nq;
    a.n_kv_heads = n_kv_heads;
    a.k = k;
    a.decay = decay;
    a.prev = prev;
    a.acc = acc;
    a.max_blocks = max_blocks;
    a.flags = flags_of(ws);
    return launch_weights_add(a, static_cast<cudaStream_t>(stream));
}

qsa_status qsa_evict_plan(const float *weights, int64_t weights_stride, const int32_t *n_tokens, int n_rows,
                          int max_blocks, int n_keep, int n_first, int n_last, int32_t *keep, int32_t *new_tokens,
                          void *ws, size_t ws_bytes, qsa_stream stream) {
    if (!weights || !n_tokens || !keep || !new_tokens)
        return fail(QSA_ERR_INVALID_ARG, "NULL weights, n_tokens, keep or new_tokens");
    if (n_rows < 1 || n_rows > (1 << 20))
        return fail(QSA_ERR_INVALID_ARG, "n_rows must be in [1, %d] (got %d)", 1 << 20, n_rows);
    if (max_blocks < 1 || max_blocks > QSA_MAX_BLOCKS)
        return fail(QSA_ERR_INVALID_ARG, "max_blocks must be in [1, %d] (got %d)", QSA_MAX_BLOCKS, max_blocks);
    if (weights_stride < max_blocks)
        return fail(QSA_ERR_INVALID_ARG, "weights_stride %lld < max_blocks %d", (long long)weights_stride, max_blocks);
    if (n_keep < 1 || n_keep > max_blocks)
        return fail(QSA_ERR_INVALID_ARG, "n_keep must be in [1, max_blocks] (got %d)", n_keep);
    if (n_first < 0 || n_last < 1 || (long long)n_first + n_last > n_keep)
        return fail(QSA_ERR_INVALID_ARG, "n_first >= 0 and n_last >= 1 must fit in n_keep (got %d, %d, %d)", n_first,
                    n_last, n_keep);
    qsa_status st = check_flags_ws(ws, ws_bytes);
    if (st != QSA_OK) return st;
    const size_t rows = (size_t)n_rows * sizeof(int32_t), keep_bytes = rows * (size_t)n_keep;
    const size_t weight_bytes = ((size_t)(n_rows - 1) * (size_t)weights_stride + (size_t)max_blocks) * sizeof(float);
    if (overlap(keep, keep_bytes, weights, weight_bytes) || overlap(keep, keep_bytes, n_tokens, rows) ||
        overlap(keep, keep_bytes, new_tokens, rows) || overlap(new_tokens, rows, weights, weight_bytes))
        return fail(QSA_ERR_INVALID_ARG, "keep and new_tokens must overlap neither each other nor an input");
    if (new_tokens != n_tokens && overlap(new_tokens, rows, n_tokens, rows))
        return fail(QSA_ERR_INVALID_ARG, "new_tokens must be n_tokens itself or not overlap it");
    EvictPlanArgs a{};
    a.weights = weights;
    a.stride = weights_stride;
    a.n_tokens = n_tokens;
    a.n_rows = n_rows;
    a.max_blocks = max_blocks;
    a.n_keep = n_keep;
    a.n_first = n_first;
    a.n_last = n_last;
    a.keep = keep;
    a.new_tokens = new_tokens;
    a.flags = flags_of(ws);
    return launch_evict_plan(a, static_cast<cudaStream_t>(stream));
}

qsa_status qsa_gather_blocks(const qsa_block_array *arrays, int n_arrays, const int32_t *keep, int n_keep, void *ws,
                             size_t ws_bytes, qsa_stream stream) {
    if (!arrays || !keep) return fail(QSA_ERR_INVALID_ARG, "NULL arrays or keep");
    if (n_arrays < 1 || n_arrays > QSA_GATHER_MAX_ARRAYS)
        return fail(QSA_ERR_INVALID_ARG, "n_arrays must be in [1, %d] (got %d)", QSA_GATHER_MAX_ARRAYS, n_arrays);
    if (n_keep < 1 || n_keep > QSA_MAX_BLOCKS)
        return fail(QSA_ERR_INVALID_ARG, "n_keep must be in [1, %d] (got %d)", QSA_MAX_BLOCKS, n_keep);
    for (int i = 0; i < n_arrays; ++i) {
        const qsa_block_array &x = arrays[i];
        if (!x.src || !x.dst) return fail(QSA_ERR_INVALID_ARG, "array %d: NULL src or dst", i);
        if (x.n_rows < 1 || x.n_rows > 65535 || x.src_blocks < 1 || x.src_blocks > QSA_MAX_BLOCKS ||
            x.dst_blocks < n_keep || x.dst_blocks > QSA_MAX_BLOCKS)
            return fail(QSA_ERR_INVALID_ARG, "array %d: bad sizes (%d rows, %d source blocks, %d destination blocks)", i,
                        x.n_rows, x.src_blocks, x.dst_blocks);
        if (x.block_bytes < 4 || x.block_bytes % 4 || x.block_bytes > (1ll << 30))
            return fail(QSA_ERR_INVALID_ARG, "array %d: block_bytes must be a multiple of 4 up to 2^30 (got %lld)", i,
                        (long long)x.block_bytes);
        if (misaligned(x.src, 4) || misaligned(x.dst, 4))
            return fail(QSA_ERR_INVALID_ARG, "array %d: src and dst must be 4-byte aligned", i);
    }
    for (int i = 0; i < n_arrays; ++i)
        for (int j = 0; j < n_arrays; ++j)
            for (int other = 0; other < 2; ++other) {   // dst i against src j, and against another dst j
                if (other && i == j) continue;
                const qsa_block_array &x = arrays[i], &y = arrays[j];
                const size_t an = (size_t)x.n_rows * x.dst_blocks * x.block_bytes;
                const size_t bn = (size_t)y.n_rows * (other ? y.dst_blocks : y.src_blocks) * y.block_bytes;
                if (overlap(x.dst, an, other ? y.dst : y.src, bn))
                    return fail(QSA_ERR_INVALID_ARG, "array %d: dst overlaps the %s of array %d", i,
                                other ? "dst" : "src", j);
            }
    qsa_status st = check_flags_ws(ws, ws_bytes);
    if (st != QSA_OK) return st;
    for (int i = 0; i < n_arrays; ++i)
        if (overlap(arrays[i].dst, (size_t)arrays[i].n_rows * arrays[i].dst_blocks * arrays[i].block_bytes, keep,
                    (size_t)n_keep * sizeof(int32_t)))
            return fail(QSA_ERR_INVALID_ARG, "array %d: dst overlaps keep", i);
    return launch_gather_blocks(arrays, n_arrays, keep, nullptr, n_keep, flags_of(ws), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
