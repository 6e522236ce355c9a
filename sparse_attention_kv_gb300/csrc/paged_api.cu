// paged_api.cu -- the C ABI of the paged 16-bit cache, of the prompt attention and of the tree attention: argument checks.
#include "qsa_internal.h"

namespace qsa {
namespace {

bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1u)) != 0; }

// A range of memory that a call reads or writes; p may be null.  An empty one overlaps nothing.
struct Range {
    const void *p;
    size_t n;
    const char *name;
};
bool overlap(const Range &a, const Range &b) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n && b.n && a0 < b0 + b.n && b0 < a0 + a.n;
}
// No output shares a byte with another output or an input.
template <int NO, int NI>
qsa_status check_apart(const Range (&out)[NO], const Range (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j])) return fail(QSA_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i], in[j])) return fail(QSA_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, in[j].name);
    }
    return QSA_OK;
}

constexpr size_t kFlagBytes = 256;   // of a workspace, in front: the flags word and what else every call keeps there
qsa_status check_ws(const void *ws, size_t ws_bytes, size_t want, bool may_be_null) {
    if (!ws && may_be_null) return QSA_OK;
    if (!ws || ws_bytes < want || misaligned(ws, 256))
        return fail(QSA_ERR_WORKSPACE, "workspace must be 256-byte aligned and hold at least %zu bytes", want);
    return QSA_OK;
}

qsa_status check_table(int64_t stride, int max_pages, int n_rows, int n_pages) {
    if (n_rows < 1 || n_rows > QSA_MAX_TABLE_ROWS)
        return fail(QSA_ERR_INVALID_ARG, "n_rows must be in [1, %d] (got %d)", QSA_MAX_TABLE_ROWS, n_rows);
    if (n_pages < 1 || n_pages > QSA_MAX_PAGES || max_pages < 1 || max_pages > QSA_MAX_PAGES)
        return fail(QSA_ERR_INVALID_ARG, "n_pages and max_pages must be in [1, %d] (got %d, %d)", QSA_MAX_PAGES, n_pages,
                    max_pages);
    if (stride < max_pages || stride > (1ll << 40))
        return fail(QSA_ERR_INVALID_ARG, "table_stride %lld < max_pages %d", (long long)stride, max_pages);
    return QSA_OK;
}
size_t table_bytes(int64_t stride, int max_pages, int n_rows) {
    return ((size_t)(n_rows - 1) * (size_t)stride + (size_t)max_pages) * sizeof(int32_t);
}
size_t words(int n) { return (size_t)n * sizeof(int32_t); }

// Rows of 128 values: what they span, given that strides are multiples of 8 and not negative.
qsa_status check_rows16(const Rows16 &x, const char *name, int tokens, int heads, long long least, size_t *bytes) {
    if (misaligned(x.p, 16)) return fail(QSA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    if (x.token % 8 || x.head % 8)
        return fail(QSA_ERR_INVALID_ARG, "%s strides must be multiples of 8 elements (got %lld, %lld)", name,
                    (long long)x.token, (long long)x.head);
    const long long most = 1ll << 38;
    if ((tokens > 1 && (x.token < least || x.token > most)) || (heads > 1 && (x.head < least || x.head > most)))
        return fail(QSA_ERR_INVALID_ARG, "%s strides must be in [%lld, 2^38] (got %lld, %lld)", name, least,
                    (long long)x.token, (long long)x.head);
    const size_t t = tokens > 1 ? (size_t)(tokens - 1) * (size_t)x.token : 0, h = heads > 1 ? (size_t)(heads - 1) * (size_t)x.head : 0;
    *bytes = tokens > 0 ? 2 * (t + h + QSA_HEAD_DIM) : 0;
    return QSA_OK;
}

PageTable page_table(const int32_t *table, int64_t stride, int max_pages, int n_rows, int n_pages, void *ws) {
    PageTable t{};
    t.table = const_cast<int32_t *>(table);
    t.stride = stride;
    t.max_pages = max_pages;
    t.n_rows = n_rows;
    t.n_pages = n_pages;
    t.flags = static_cast<uint32_t *>(ws);
    return t;
}

size_t pages_ws_bytes(int n_rows, int n_pages) {
    return 256 + ((size_t)n_rows + (size_t)n_pages + 1 + 63) / 64 * 256;
}
PagesWs pages_ws(void *ws, int n_rows, int n_pages) {
    PagesWs w{};
    w.upto = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + 256);
    w.list = w.upto + n_rows;
    w.live = w.list + n_pages;
    return w;
}

// What both attentions check: types, heads, rows and outputs; in and out ranges for check_apart.
qsa_status check_dense(const DenseArgs &a, int head_dim, size_t ws_bytes, size_t (&spans)[3]) {
    if (!a.q.p || !a.k.p || !a.v.p || !a.cu_q || !a.out) return fail(QSA_ERR_INVALID_ARG, "NULL q, k, v, cu or out");
    if (a.dt != QSA_BF16 && a.dt != QSA_F16)
        return fail(QSA_ERR_UNSUPPORTED, "the attention takes bf16 or fp16 (dtype %d)", (int)a.dt);
    if (head_dim != QSA_HEAD_DIM)
        return fail(QSA_ERR_INVALID_ARG, "head_dim must be %d (got %d)", QSA_HEAD_DIM, head_dim);
    if (a.n_kv_heads < 1 || a.n_kv_heads > 65535 || a.n_heads < 1 || a.n_heads % a.n_kv_heads ||
        a.n_heads / a.n_kv_heads > QSA_ATTN_GROUP)
        return fail(QSA_ERR_INVALID_ARG, "n_heads must be 1 to %d times n_kv_heads in [1, 65535] (got %d heads, %d KV heads)",
                    QSA_ATTN_GROUP, a.n_heads, a.n_kv_heads);
    if (a.n_seqs < 1 || a.n_seqs > 65535) return fail(QSA_ERR_INVALID_ARG, "n_seqs must be in [1, 65535] (got %d)", a.n_seqs);
    if (a.total_q < 0 || a.total_k < 0 || (long long)a.total_q * a.n_heads >= (1ll << 30) || a.total_k >= (1 << 30))
        return fail(QSA_ERR_INVALID_ARG, "rows out of range (%d queries, %d keys)", a.total_q, a.total_k);
    if (!(a.scale > 0.0f) || !(a.scale <= 3.4e38f)) return fail(QSA_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (a.out_dt != QSA_F32 && a.out_dt != a.dt)
        return fail(QSA_ERR_INVALID_ARG, "out must be fp32 or of the inputs' dtype (got %d)", (int)a.out_dt);
    if (misaligned(a.out, 16)) return fail(QSA_ERR_INVALID_ARG, "out must be 16-byte aligned");
    qsa_status st;
    if ((st = check_rows16(a.q, "q", a.total_q, a.n_heads, 0, &spans[0])) != QSA_OK ||
        (st = check_rows16(a.k, "k", a.total_k, a.n_kv_heads, QSA_HEAD_DIM, &spans[1])) != QSA_OK ||
        (st = check_rows16(a.v, "v", a.total_k, a.n_kv_heads, QSA_HEAD_DIM, &spans[2])) != QSA_OK)
        return st;
    return check_ws(a.ws, ws_bytes, attention_ws_bytes(a.total_q > 0 ? a.total_q : 1, a.n_heads, a.n_kv_heads), false);
}
size_t out_bytes(const DenseArgs &a) {
    return (size_t)a.total_q * a.n_heads * QSA_HEAD_DIM * (a.out_dt == QSA_F32 ? 4 : 2);
}

// a: everything but the pool and the table.
qsa_status pages_append(const PagesAppendArgs &a, qsa_dtype dt, const int32_t *table, int64_t table_stride, int max_pages,
                        int n_rows, int head_dim, int capacity, void *ws, size_t ws_bytes, qsa_stream stream) {
    if (!a.k.p || !a.v.p || !a.cu_rows || !a.first || !table || !a.kcache || !a.vcache_t)
        return fail(QSA_ERR_INVALID_ARG, "NULL k, v, cu_rows, first, table, kcache or vcache_t");
    if (dt != QSA_BF16 && dt != QSA_F16)
        return fail(QSA_ERR_UNSUPPORTED, "the paged cache takes bf16 or fp16 rows (dtype %d)", (int)dt);
    if (head_dim != QSA_HEAD_DIM)
        return fail(QSA_ERR_INVALID_ARG, "head_dim must be %d (got %d)", QSA_HEAD_DIM, head_dim);
    if (a.n_kv_heads < 1 || a.n_kv_heads > 65535)
        return fail(QSA_ERR_INVALID_ARG, "n_kv_heads must be in [1, 65535] (got %d)", a.n_kv_heads);
    if (capacity < 64 || capacity % 64)
        return fail(QSA_ERR_INVALID_ARG, "capacity must be a positive multiple of 64 (got %d)", capacity);
    qsa_status st = check_table(table_stride, max_pages, n_rows, capacity / 64);
    if (st != QSA_OK) return st;
    if (a.n < 0 || a.n > (1 << 28) || a.n_source < 0 || a.n_source > (1 << 28) || (!a.rows && a.n != a.n_source))
        return fail(QSA_ERR_INVALID_ARG, "bad numbers of rows (%d entries, %d rows)", a.n, a.n_source);
    size_t kb, vb;
    if ((st = check_rows16(a.k, "k", a.n_source, a.n_kv_heads, 0, &kb)) != QSA_OK ||
        (st = check_rows16(a.v, "v", a.n_source, a.n_kv_heads, 0, &vb)) != QSA_OK)
        return st;
    if (misaligned(a.kcache, 16) || misaligned(a.vcache_t, 16))
        return fail(QSA_ERR_INVALID_ARG, "kcache and vcache_t must be 16-byte aligned");
    if ((st = check_ws(ws, ws_bytes, kFlagBytes, true)) != QSA_OK) return st;
    const size_t pool = (size_t)a.n_kv_heads * capacity * QSA_HEAD_DIM * 2;
    const Range out[] = {{a.kcache, pool, "kcache"}, {a.vcache_t, pool, "vcache_t"}, {ws, kFlagBytes, "ws"}};
    const Range in[] = {{a.k.p, kb, "k"}, {a.v.p, vb, "v"}, {a.rows, words(a.n), "rows"}, {a.cu_rows, words(n_rows + 1), "cu_rows"},
                        {a.first, words(n_rows), "first"}, {a.end, words(n_rows), "end"},
                        {table, table_bytes(table_stride, max_pages, n_rows), "table"}};
    if ((st = check_apart(out, in)) != QSA_OK) return st;
    if (a.n == 0) return QSA_OK;
    return launch_pages_append(page_table(table, table_stride, max_pages, n_rows, capacity / 64, ws), a,
                               static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace qsa

using namespace qsa;

extern "C" {

size_t qsa_pages_workspace_bytes(int n_rows, int n_pages) {
    if (n_rows < 1 || n_rows > QSA_MAX_TABLE_ROWS || n_pages < 1 || n_pages > QSA_MAX_PAGES) return 0;
    return pages_ws_bytes(n_rows, n_pages);
}

qsa_status qsa_pages_fork(int32_t *table, int64_t table_stride, int max_pages, int32_t *n_tokens, int n_rows,
                          int32_t *refs, int n_pages, const int32_t *src, const int32_t *dst, int n, void *ws,
                          size_t ws_bytes, qsa_stream stream) {
    if (!table || !n_tokens || !refs || !src || !dst)
        return fail(QSA_ERR_INVALID_ARG, "NULL table, n_tokens, refs, src or dst");
    qsa_status st = check_table(table_stride, max_pages, n_rows, n_pages);
    if (st != QSA_OK) return st;
    if (n < 0 || n > n_rows) return fail(QSA_ERR_INVALID_ARG, "n must be in [0, n_rows] (got %d)", n);
    if ((st = check_ws(ws, ws_bytes, kFlagBytes, true)) != QSA_OK) return st;
    const Range out[] = {{table, table_bytes(table_stride, max_pages, n_rows), "table"}, {n_tokens, words(n_rows), "n_tokens"},
                         {refs, words(n_pages), "refs"}, {ws, kFlagBytes, "ws"}};
    const Range in[] = {{src, words(n), "src"}, {dst, words(n), "dst"}};
    if ((st = check_apart(out, in)) != QSA_OK) return st;
    if (n == 0) return QSA_OK;
    return launch_pages_fork(page_table(table, table_stride, max_pages, n_rows, n_pages, ws), n_tokens, refs, src, dst, n,
                             static_cast<cudaStream_t>(stream));
}

qsa_status qsa_pages_release(int32_t *table, int64_t table_stride, int max_pages, int32_t *n_tokens, int n_rows,
                             int32_t *refs, int n_pages, const int32_t *keep, void *ws, size_t ws_bytes,
                             qsa_stream stream) {
    if (!table || !n_tokens || !refs || !keep) return fail(QSA_ERR_INVALID_ARG, "NULL table, n_tokens, refs or keep");
    qsa_status st = check_table(table_stride, max_pages, n_rows, n_pages);
    if (st != QSA_OK || (st = check_ws(ws, ws_bytes, kFlagBytes, true)) != QSA_OK) return st;
    const Range out[] = {{table, table_bytes(table_stride, max_pages, n_rows), "table"}, {n_tokens, words(n_rows), "n_tokens"},
                         {refs, words(n_pages), "refs"}, {ws, kFlagBytes, "ws"}};
    const Range in[] = {{keep == n_tokens ? nullptr : keep, words(n_rows), "keep"}};
    if ((st = check_apart(out, in)) != QSA_OK) return st;
    return launch_pages_release(page_table(table, table_stride, max_pages, n_rows, n_pages, ws), n_tokens, refs, keep,
                                static_cast<cudaStream_t>(stream));
}

qsa_status qsa_pages_reserve(int32_t *table, int64_t table_stride, int max_pages, const int32_t *n_tokens, int n_rows,
                             int32_t *refs, int n_pages, const int32_t *add, int32_t *new_tokens, int32_t *copy_src,
                             int32_t *copy_dst, void *ws, size_t ws_bytes, qsa_stream stream) {
    if (!table || !n_tokens || !refs || !add || !new_tokens || !copy_src || !copy_dst)
        return fail(QSA_ERR_INVALID_ARG, "NULL table, n_tokens, refs, add, new_tokens, copy_src or copy_dst");
    qsa_status st = check_table(table_stride, max_pages, n_rows, n_pages);
    if (st != QSA_OK || (st = check_ws(ws, ws_bytes, pages_ws_bytes(n_rows, n_pages), false)) != QSA_OK) return st;
    const Range out[] = {{table, table_bytes(table_stride, max_pages, n_rows), "table"}, {refs, words(n_pages), "refs"},
                         {new_tokens, words(n_rows), "new_tokens"}, {copy_src, words(n_rows), "copy_src"},
                         {copy_dst, words(n_rows), "copy_dst"}, {ws, pages_ws_bytes(n_rows, n_pages), "ws"}};
    const Range in[] = {{n_tokens, words(n_rows), "n_tokens"}, {add, words(n_rows), "add"}};
    if ((st = check_apart(out, in)) != QSA_OK) return st;
    return launch_pages_reserve(page_table(table, table_stride, max_pages, n_rows, n_pages, ws), n_tokens, refs, add,
                                new_tokens, copy_src, copy_dst, pages_ws(ws, n_rows, n_pages),
                                static_cast<cudaStream_t>(stream));
}

qsa_status qsa_pages_compact(const int32_t *table, int64_t table_stride, int max_pages, int n_rows, const int32_t *refs,
                             int n_pages, int32_t *table_out, int32_t *refs_out, int32_t *copy_src, int32_t *copy_dst,
                             void *ws, size_t ws_bytes, qsa_stream stream) {
    if (!table || !refs || !table_out || !refs_out || (n_pages > 1 && (!copy_src || !copy_dst)))
        return fail(QSA_ERR_INVALID_ARG, "NULL table, refs, table_out, refs_out, copy_src or copy_dst");
    qsa_status st = check_table(table_stride, max_pages, n_rows, n_pages);
    if (st != QSA_OK || (st = check_ws(ws, ws_bytes, pages_ws_bytes(n_rows, n_pages), false)) != QSA_OK) return st;
    const size_t tb = table_bytes(table_stride, max_pages, n_rows);
    const Range out[] = {{table_out, tb, "table_out"}, {refs_out, words(n_pages), "refs_out"},
                         {copy_src, words(n_pages / 2), "copy_src"}, {copy_dst, words(n_pages / 2), "copy_dst"},
                         {ws, pages_ws_bytes(n_rows, n_pages), "ws"}};
    const Range in[] = {{table == table_out ? nullptr : table, tb, "table"},
                        {refs == refs_out ? nullptr : refs, words(n_pages), "refs"}};
    if ((st = check_apart(out, in)) != QSA_OK) return st;
    return launch_pages_compact(page_table(table, table_stride, max_pages, n_rows, n_pages, ws), refs, table_out, refs_out,
                                copy_src, copy_dst, pages_ws(ws, n_rows, n_pages), static_cast<cudaStream_t>(stream));
}

qsa_status qsa_pages_copy(const qsa_block_array *arrays, int n_arrays, const int32_t *src_ids, const int32_t *dst_ids,
                          int n, void *ws, size_t ws_bytes, qsa_stream stream) {
    if (!arrays || !src_ids || !dst_ids) return fail(QSA_ERR_INVALID_ARG, "NULL arrays, src_ids or dst_ids");
    if (n_arrays < 1 || n_arrays > QSA_GATHER_MAX_ARRAYS)
        return fail(QSA_ERR_INVALID_ARG, "n_arrays must be in [1, %d] (got %d)", QSA_GATHER_MAX_ARRAYS, n_arrays);
    if (n < 0 || n > QSA_MAX_PAGES) return fail(QSA_ERR_INVALID_ARG, "n must be in [0, %d] (got %d)", QSA_MAX_PAGES, n);
    qsa_status st = check_ws(ws, ws_bytes, kFlagBytes, true);
    if (st != QSA_OK) return st;
    const Range flags[] = {{ws, kFlagBytes, "ws"}};
    const Range ids[] = {{src_ids, words(n), "src_ids"}, {dst_ids, words(n), "dst_ids"}};
    if ((st = check_apart(flags, ids)) != QSA_OK) return st;
    for (int i = 0; i < n_arrays; ++i) {
        const qsa_block_array &x = arrays[i];
        if (!x.dst || x.src != x.dst) return fail(QSA_ERR_INVALID_ARG, "array %d: src must be dst, the pool", i);
        if (x.n_rows < 1 || x.n_rows > 65535 || x.dst_blocks < 1 || x.dst_blocks > QSA_MAX_PAGES || x.src_blocks != x.dst_blocks)
            return fail(QSA_ERR_INVALID_ARG, "array %d: bad sizes (%d rows, %d and %d pages)", i, x.n_rows, x.src_blocks,
                        x.dst_blocks);
        if (x.block_bytes < 4 || x.block_bytes % 4 || x.block_bytes > (1ll << 30))
            return fail(QSA_ERR_INVALID_ARG, "array %d: block_bytes must be a multiple of 4 up to 2^30 (got %lld)", i,
                        (long long)x.block_bytes);
        if (misaligned(x.dst, 4)) return fail(QSA_ERR_INVALID_ARG, "array %d: must be 4-byte aligned", i);
        const Range pool[] = {{x.dst, (size_t)x.n_rows * x.dst_blocks * x.block_bytes, "an array"}};
        if ((st = check_apart(pool, ids)) != QSA_OK || (st = check_apart(pool, flags)) != QSA_OK) return st;
        for (int j = 0; j < i; ++j) {
            const qsa_block_array &y = arrays[j];
            const Range other[] = {{y.dst, (size_t)y.n_rows * y.dst_blocks * y.block_bytes, "another one"}};
            if (overlap(pool[0], other[0])) return fail(QSA_ERR_INVALID_ARG, "array %d overlaps array %d", i, j);
        }
    }
    if (n == 0) return QSA_OK;
    return launch_gather_blocks(arrays, n_arrays, src_ids, dst_ids, n, static_cast<uint32_t *>(ws),
                                static_cast<cudaStream_t>(stream));
}

qsa_status qsa_pages_append(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                            int64_t v_token_stride, int64_t v_head_stride, qsa_dtype dt, int n_source,
                            const int32_t *rows, int n, const int32_t *cu_rows, const int32_t *first,
                            const int32_t *table, int64_t table_stride, int max_pages, int n_rows, int n_kv_heads,
                            int head_dim, void *kcache, void *vcache_t, int capacity, void *ws, size_t ws_bytes,
                            qsa_stream stream) {
    const PagesAppendArgs a{{k, k_token_stride, k_head_stride}, {v, v_token_stride, v_head_stride}, n_source, rows, n, cu_rows,
                            first, nullptr, n_kv_heads, kcache, vcache_t};
    return pages_append(a, dt, table, table_stride, max_pages, n_rows, head_dim, capacity, ws, ws_bytes, stream);
}

qsa_status qsa_pages_append_reserved(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                                     int64_t v_token_stride, int64_t v_head_stride, qsa_dtype dt, int n_source,
                                     const int32_t *rows, int n, const int32_t *cu_rows, const int32_t *first,
                                     const int32_t *end, const int32_t *table, int64_t table_stride, int max_pages,
                                     int n_rows, int n_kv_heads, int head_dim, void *kcache, void *vcache_t,
                                     int capacity, void *ws, size_t ws_bytes, qsa_stream stream) {
    if (!end) return fail(QSA_ERR_INVALID_ARG, "NULL end");
    const PagesAppendArgs a{{k, k_token_stride, k_head_stride}, {v, v_token_stride, v_head_stride}, n_source, rows, n, cu_rows,
                            first, end, n_kv_heads, kcache, vcache_t};
    return pages_append(a, dt, table, table_stride, max_pages, n_rows, head_dim, capacity, ws, ws_bytes, stream);
}

size_t qsa_attention_workspace_bytes(int rows, int n_heads, int n_kv_heads) {
    if (rows < 1 || n_kv_heads < 1 || n_kv_heads > 65535 || n_heads < 1 || n_heads % n_kv_heads ||
        n_heads / n_kv_heads > QSA_ATTN_GROUP || (long long)rows * n_heads >= (1ll << 30))
        return 0;
    return attention_ws_bytes(rows, n_heads, n_kv_heads);
}

qsa_status qsa_prompt_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                                int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                                int64_t v_head_stride, qsa_dtype dt, const int32_t *cu_q, const int32_t *cu_k, int n_seqs,
                                int total_q, int total_k, int n_heads, int n_kv_heads, int head_dim, float scale,
                                void *out, qsa_dtype out_dt, float *lse, void *ws, size_t ws_bytes, qsa_stream stream) {
    DenseArgs a{};
    a.dt = dt;
    a.q = {q, q_token_stride, q_head_stride};
    a.k = {k, k_token_stride, k_head_stride};
    a.v = {v, v_token_stride, v_head_stride};
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.n_seqs = n_seqs;
    a.total_q = total_q;
    a.total_k = total_k;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.scale = scale;
    a.out = out;
    a.out_dt = out_dt;
    a.lse = lse;
    a.ws = ws;
    a.flags = static_cast<uint32_t *>(ws);
    size_t spans[3];
    if (!cu_k) return fail(QSA_ERR_INVALID_ARG, "NULL cu_k");
    qsa_status st = check_dense(a, head_dim, ws_bytes, spans);
    if (st != QSA_OK) return st;
    const Range outs[] = {{out, out_bytes(a), "out"}, {lse, (size_t)total_q * n_heads * 4, "lse"}, {ws, ws_bytes, "ws"}};
    const Range ins[] = {{q, spans[0], "q"}, {k, spans[1], "k"}, {v, spans[2], "v"}, {cu_q, words(n_seqs + 1), "cu_q"},
                         {cu_k, words(n_seqs + 1), "cu_k"}};
    if ((st = check_apart(outs, ins)) != QSA_OK || total_q == 0) return st;
    return launch_prompt_attention(a, static_cast<cudaStream_t>(stream));
}

qsa_status qsa_tree_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                              int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                              int64_t v_head_stride, qsa_dtype dt, const int32_t *parents, const int32_t *cu_nodes,
                              int n_seqs, int total_nodes, int max_nodes, const void *kcache, const void *vcache_t,
                              int capacity, const int32_t *table, int64_t table_stride, int max_pages,
                              const int32_t *n_tokens, int n_heads, int n_kv_heads, int head_dim, float scale,
                              void *out, qsa_dtype out_dt, float *lse, void *ws, size_t ws_bytes, qsa_stream stream) {
    DenseArgs a{};
    a.dt = dt;
    a.q = {q, q_token_stride, q_head_stride};
    a.k = {k, k_token_stride, k_head_stride};
    a.v = {v, v_token_stride, v_head_stride};
    a.cu_q = cu_nodes;
    a.n_seqs = n_seqs;
    a.total_q = a.total_k = total_nodes;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.scale = scale;
    a.out = out;
    a.out_dt = out_dt;
    a.lse = lse;
    a.parents = parents;
    a.max_nodes = max_nodes;
    a.kcache = kcache;
    a.vcache_t = vcache_t;
    a.n_tokens = n_tokens;
    a.ws = ws;
    a.flags = static_cast<uint32_t *>(ws);
    if (!parents || !kcache || !vcache_t || !table || !n_tokens)
        return fail(QSA_ERR_INVALID_ARG, "NULL parents, kcache, vcache_t, table or n_tokens");
    size_t spans[3];
    qsa_status st = check_dense(a, head_dim, ws_bytes, spans);
    if (st != QSA_OK) return st;
    if (max_nodes < 1 || max_nodes > QSA_TREE_MAX_NODES)
        return fail(QSA_ERR_INVALID_ARG, "max_nodes must be in [1, %d] (got %d)", QSA_TREE_MAX_NODES, max_nodes);
    if (capacity < 64 || capacity % 64 || capacity / 64 > QSA_MAX_PAGES || (long long)n_kv_heads * capacity >= (1ll << 30))
        return fail(QSA_ERR_INVALID_ARG, "capacity must be a positive multiple of 64 of at most %d pages, below 2^30 with all heads (got %d)",
                    QSA_MAX_PAGES, capacity);
    if (max_pages < 1 || max_pages > QSA_MAX_PAGES || table_stride < max_pages || table_stride > (1ll << 40))
        return fail(QSA_ERR_INVALID_ARG, "max_pages must be in [1, %d] and table_stride no less (got %d, %lld)", QSA_MAX_PAGES,
                    max_pages, (long long)table_stride);
    if (misaligned(kcache, 16) || misaligned(vcache_t, 16))
        return fail(QSA_ERR_INVALID_ARG, "kcache and vcache_t must be 16-byte aligned");
    a.table = page_table(table, table_stride, max_pages, n_seqs, capacity / 64, ws);
    const size_t pool = (size_t)n_kv_heads * capacity * QSA_HEAD_DIM * 2;
    const Range outs[] = {{out, out_bytes(a), "out"}, {lse, (size_t)total_nodes * n_heads * 4, "lse"}, {ws, ws_bytes, "ws"}};
    const Range ins[] = {{q, spans[0], "q"}, {k, spans[1], "k"}, {v, spans[2], "v"}, {cu_nodes, words(n_seqs + 1), "cu_nodes"},
                         {parents, words(total_nodes), "parents"}, {kcache, pool, "kcache"}, {vcache_t, pool, "vcache_t"},
                         {table, table_bytes(table_stride, max_pages, n_seqs), "table"}, {n_tokens, words(n_seqs), "n_tokens"}};
    if ((st = check_apart(outs, ins)) != QSA_OK || total_nodes == 0) return st;
    return launch_tree_attention(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
