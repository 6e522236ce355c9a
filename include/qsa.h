/*
 * qsa.h -- C ABI of the GB300 (sm_103a) query-sparse-attention block selection
 * library, libqsa.so.
 *
 * The path selects, for every query, the KV blocks (64 tokens each) that a
 * sparse attention step will read:
 *
 *   1. block scorer:  score[q][b] = sum_h w[q][h] * relu(dot(q[q][h][:], kblk[b][:]))
 *      over the indexer heads h, head dim 128, one key row per block (the last,
 *      partial block of a context has a key like any other);
 *   2. block top-k:   the k blocks of highest score, ties to the lower block id,
 *      emitted as ids in ascending block order, -1 padded when n < k.
 *
 * Sources: the scorer is the "qsa_block_scores" step of "#1091 qsa_select:
 * FP32 tiled block scores below sm_80" (section "What": rows = query x indexer
 * head, K = 128, ReLU per head summed per block; the tail block).  The top-k
 * rule is the threshold / "above" / tie-budget rule of "#2093 sm_75: the
 * prompt path's top-k with one full read of the scores" (description, steps
 * 1-4), and the decode split is the two-stage split of Strata PR #3987
 * (section "Approach").
 *
 * Conventions for every entry point:
 *  - Every pointer argument except the ones marked "host" is DEVICE memory owned
 *    by the caller.  The library never allocates or frees memory on a call and
 *    never synchronises the device.  Scratch lives in the caller's workspace, with
 *    one exception: qsa_block_topk_static uses a fixed scratch array compiled into
 *    the library (see there); no other entry point keeps device state between calls.
 *  - Work is enqueued on `stream` (a cudaStream_t, NULL = legacy default stream)
 *    and runs asynchronously; the return value reports host-side validation and
 *    launch errors only.  Device-side contract violations are recorded as bits in
 *    the workspace flags word (QSA_FLAG_*), readable with qsa_read_flags().
 *  - On any error status nothing is enqueued; qsa_last_error() (thread-local)
 *    returns a one-line reason.
 *  - One workspace must not be used by two calls that can run concurrently
 *    (e.g. on two streams); give each stream its own workspace.
 *  - An output overlaps neither an input nor another output, unless its call says
 *    that it may.
 */
#ifndef QSA_H
#define QSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QSA_VERSION 1

/* Head dimension of q and kblk rows; the only value supported. */
#define QSA_HEAD_DIM 128
/* Largest k (blocks selected per query). */
#define QSA_MAX_K 1024
/* Largest max_blocks (KV capacity in blocks). */
#define QSA_MAX_BLOCKS (1 << 24)

typedef enum {
    QSA_OK = 0,
    QSA_ERR_INVALID_ARG = 1, /* bad pointer, size, alignment or enum value */
    QSA_ERR_UNSUPPORTED = 2, /* a forced path that cannot run this shape */
    QSA_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than qsa_workspace_bytes() */
    QSA_ERR_CUDA = 4         /* a CUDA runtime/driver call or a launch failed */
} qsa_status;

typedef enum {
    QSA_F32 = 0,  /* IEEE binary32 */
    QSA_BF16 = 1, /* bfloat16 (upper half of a binary32) */
    QSA_E4M3 = 2, /* 8-bit floating point E4M3 of the OCP FP8 specification (sign, 4 exponent bits
                     with bias 7, 3 mantissa bits; no infinities, S.1111.111 = NaN) */
    QSA_F16 = 3   /* IEEE binary16 (qsa_select_attention only) */
} qsa_dtype;

/* Top-k path.  AUTO picks from host-visible sizes only; the others force a path
 * (tests).  Every path returns the same ids. */
typedef enum {
    QSA_PATH_AUTO = 0,
    QSA_PATH_SPLIT = 1,    /* multi-CTA chunk split + last-CTA merge (decode windows) */
    QSA_PATH_SAMPLE = 2,   /* one read against a sampled lower bound (+ radix fallback) */
    QSA_PATH_REGISTER = 3, /* whole row in registers, one CTA per query */
    QSA_PATH_RADIX = 4,    /* multi-pass radix select over global memory, any size */
    QSA_PATH_WARP = 5      /* k <= 32, rows of up to 8,192 blocks held in registers (one warp per
                              1,024): a bound from the row's lane maxima keeps a few more than k
                              scores, which are ranked exactly; heavy ties take a per-chunk select
                              and merge */
} qsa_path;

typedef void *qsa_stream; /* a cudaStream_t */

/* Bits of the workspace flags word (sticky until cleared by qsa_read_flags). */
#define QSA_FLAG_NBLOCKS_CLAMPED 0x1u /* some n_blocks[q] was < 0 or > its bound; clamped */
#define QSA_FLAG_WAIT_TIMEOUT 0x2u    /* a kernel gave up a bounded wait; its outputs are invalid */
#define QSA_FLAG_INTERNAL 0x4u        /* an internal consistency check failed */
#define QSA_FLAG_SAMPLE_FALLBACK 0x8u /* not an error: some query of the sampled filter had too few
                                         or too many candidates and was selected from its whole row */
#define QSA_FLAG_BAD_ID 0x10u         /* a call skipped an id outside its range (an id other than -1):
                                         a query's context in the attentions, max_blocks or the
                                         source's blocks elsewhere */
#define QSA_FLAG_BAD_WEIGHT 0x20u     /* qsa_block_weights_add met a weight outside
                                         [0, QSA_MAX_BLOCK_WEIGHT] or a NaN; it was clamped (NaN: 0) */

/* Query heads per KV head (GQA group) of qsa_select_attention. */
#define QSA_ATTN_GROUP 16
/* Largest k of qsa_select_attention. */
#define QSA_ATTN_MAX_K 64

/*
 * Workspace size in bytes for calls with these sizes: fused != 0 for the fused
 * form of qsa_select (its per-CTA candidate lists take up to 4,096 entries per
 * query), else any other call.  A workspace sized for (nq, max_blocks, k, fused)
 * serves every call with sizes at or below these.  The workspace must be zero-filled before its first use (e.g. by
 * qsa_workspace_init); every call leaves it in a reusable state.  Returns 0 for
 * invalid sizes.
 */
size_t qsa_workspace_bytes(int nq, int max_blocks, int k, int fused);

/* Zero-fill `ws_bytes` bytes of workspace `ws` on `stream` (cudaMemsetAsync). */
qsa_status qsa_workspace_init(void *ws, size_t ws_bytes, qsa_stream stream);

/*
 * Block scores: scores[q * scores_stride + b] for 0 <= b < n_blocks[q].
 *
 *   q        [nq][n_heads][128]  dtype `dt` (fp32, bf16 or fp8 e4m3), row-major, 16-byte aligned
 *   w        [nq][n_heads]       fp32
 *   kblk     [max_blocks][128]   dtype `dt`, row-major, 16-byte aligned
 *   n_blocks [nq]                int32 on the DEVICE: blocks in each query's context,
 *                                clamped on the device to [0, bound] where bound =
 *                                active_blocks if active_blocks >= 0, else max_blocks
 *                                (a clamp sets QSA_FLAG_NBLOCKS_CLAMPED)
 *   active_blocks                host int: -1 (unknown) or an upper bound on every
 *                                n_blocks[q] (values above max_blocks act as max_blocks);
 *                                it sizes the grid and never changes a result
 *   scores   [nq][scores_stride] fp32, scores_stride >= max_blocks; entries at
 *                                b >= n_blocks[q] are not written
 *   ws, ws_bytes                 workspace (may be NULL/0: then device flags are not
 *                                recorded)
 *
 * Arithmetic: products on the tensor cores (bf16 x bf16 -> fp32, e4m3 x e4m3 ->
 * fp32, or fp32 split in three tf32 products), accumulated in fp32; ReLU and the
 * head-weighted sum in fp32.  n_heads must be 1, 2, 4, 8 or 16.  e4m3 stores the
 * indexer keys (and queries) in 8 bits, as the pages' engine stores its KV cache
 * in 8 bits ("--kv int8"); the tensor-core 8-bit format of this GPU is e4m3.
 * Launch: the kernel is launched as a programmatic dependent of the work before it
 * on `stream`: its CTAs may be scheduled while that work drains, and wait at entry,
 * before they take tensor memory or touch any buffer, until it has completed.
 * Errors: QSA_ERR_INVALID_ARG for NULL q/w/kblk/n_blocks/scores, nq < 1,
 * head_dim != 128, unsupported n_heads, max_blocks outside [1, QSA_MAX_BLOCKS],
 * scores_stride < max_blocks, misaligned q/kblk, a dtype other than QSA_F32,
 * QSA_BF16 or QSA_E4M3.
 */
qsa_status qsa_block_scores(const void *q, const float *w, const void *kblk, qsa_dtype dt,
                            const int32_t *n_blocks, int nq, int n_heads, int head_dim,
                            int max_blocks, int active_blocks, float *scores,
                            int64_t scores_stride, void *ws, size_t ws_bytes, qsa_stream stream);

/*
 * Block top-k over given fp32 scores.
 *
 *   scores   [nq][scores_stride] fp32 (NaN is outside the contract; -0 == +0); every
 *            entry below the bound (active_blocks, else max_blocks) must be readable
 *            memory: entries at or past n_blocks[q] may be read but never affect ids
 *   n_blocks [nq] int32 on the DEVICE, clamped as for qsa_block_scores
 *   k        1 <= k <= QSA_MAX_K
 *   ids      [nq][k] int32 out: the selected block ids in ascending order; when
 *            n_blocks[q] < k the first n_blocks[q] slots hold 0..n-1 and the rest -1
 *   ws       workspace of at least qsa_workspace_bytes(nq, max_blocks, k, 0) bytes
 *   path     QSA_PATH_AUTO, or a forced path (QSA_ERR_UNSUPPORTED if it cannot run
 *            this shape)
 *
 * Selection: keep the blocks that come first in the order (score descending,
 * block id ascending).  Every path gives the same ids.
 */
qsa_status qsa_block_topk(const float *scores, int64_t scores_stride, const int32_t *n_blocks,
                          int nq, int max_blocks, int active_blocks, int k, int32_t *ids,
                          void *ws, size_t ws_bytes, qsa_path path, qsa_stream stream);

/*
 * Block top-k for callers that cannot allocate device memory.  No passage of the
 * source pages has a counterpart to this call; it exists for callers that may
 * not call cudaMalloc where they select blocks (a fixed memory arena that must
 * not grow, a plug-in given only its input and output buffers, a serving path
 * where device allocation is forbidden).
 *
 * Same arguments, results and errors as qsa_block_topk, without ws / ws_bytes:
 * the scratch is an 8 MiB array compiled into the library, held on every GPU
 * that loads it until the process exits.  Sizes whose workspace
 * (qsa_workspace_bytes(nq, max_blocks, k, 0)) exceeds 8 MiB are rejected with
 * QSA_ERR_WORKSPACE and nothing is launched.  The call never allocates.
 *
 * The first call on each device looks up the scratch's device address (a CUDA
 * runtime query, with that device current) and caches it, and looks it up again
 * when the device's context has been replaced (after cudaDeviceReset); make that
 * first call before any stream capture.  A call rejected by its argument checks
 * enqueues nothing, not even the clear below.  All calls share the one scratch array: the parts
 * that must start at zero are cleared on `stream` at the start of every call,
 * and calls that can overlap on the GPU (different streams or host threads)
 * race with each other.  The device flags of these calls are not readable.
 */
qsa_status qsa_block_topk_static(const float *scores, int64_t scores_stride, const int32_t *n_blocks, int nq,
                                 int max_blocks, int active_blocks, int k, int32_t *ids, qsa_path path,
                                 qsa_stream stream);

/*
 * KV-sharded selection, stage A: the candidates of one shard of the KV blocks.
 * A query's selection restricted to a subset of its blocks is a prefix of that
 * subset's selection order (score descending, block id ascending), so the k best
 * blocks of every shard, merged by qsa_merge_candidates, select exactly the blocks
 * one call over all of them selects (Strata PR #3987, section "Approach": each
 * chunk keeps its top k, one CTA per query selects over the union).  The shards
 * may live on different GPUs: each computes its candidates, an all-gather collects
 * nq x k of them per shard, and every GPU merges.
 *
 *   scores, scores_stride, n_blocks, nq, max_blocks, active_blocks, k, ws, ws_bytes,
 *   path           as for qsa_block_topk, over this shard's blocks (local ids 0 ..
 *                  n_blocks[q] - 1)
 *   block_offset   host int: the global id of the shard's first block; ids
 *                  block_offset + max_blocks - 1 must stay below 2^31 - 1
 *   cand_ids       [nq][k] int32 out: the shard's selection as global ids
 *                  (block_offset + local id), ascending, -1 padded when n_blocks[q] < k
 *   cand_scores    [nq][k] fp32 out: each candidate's score (-inf where the id is -1)
 *
 * Two launches on `stream`: the top-k (any path) into cand_ids, then a kernel that
 * reads the candidates' scores and offsets their ids.
 * Errors: as qsa_block_topk, plus QSA_ERR_INVALID_ARG for NULL cand_scores /
 * cand_ids or a block_offset outside the range above.
 */
qsa_status qsa_block_candidates(const float *scores, int64_t scores_stride, const int32_t *n_blocks, int nq,
                                int max_blocks, int active_blocks, int k, int32_t block_offset, float *cand_scores,
                                int32_t *cand_ids, void *ws, size_t ws_bytes, qsa_path path, qsa_stream stream);

/*
 * KV-sharded selection, stage B: the k blocks of highest score over every shard's
 * candidates, ties to the lower global id, emitted as ids in ascending order (-1
 * padded when all shards together hold fewer than k candidates).
 *
 *   cand_scores  [n_shards][nq][k] fp32: the shards' qsa_block_candidates outputs,
 *                shard-major (the layout an all-gather of the [nq][k] arrays leaves)
 *   cand_ids     [n_shards][nq][k] int32: their global ids; entries < 0 are empty;
 *                the shards' ids must be distinct (disjoint block ranges)
 *   ids          [nq][k] int32 out
 *
 * One launch (one CTA per query), no workspace.
 * Errors: QSA_ERR_INVALID_ARG for NULL pointers, nq < 1, k outside [1, QSA_MAX_K],
 * n_shards < 1, n_shards x nq x k >= 2^31; QSA_ERR_UNSUPPORTED when n_shards x k
 * exceeds 4,096 candidates per query.
 */
qsa_status qsa_merge_candidates(const float *cand_scores, const int32_t *cand_ids, int n_shards, int nq, int k,
                                int32_t *ids, qsa_stream stream);

/*
 * Score then select, in one call.
 *
 * fused == 0 (chained): the scorer writes `scores` (required), then the top-k
 *   reads them; both are the calls above.
 * fused != 0: the scores never go to HBM.  The scorer keeps each CTA's block
 *   range of scores on chip and, per query, one warp lists every block of that
 *   range that can be in the selection (the scores at or above the k-th largest
 *   lane maximum for k <= 32, else the range's exact top k) in the workspace with
 *   the list's length; a merge kernel, launched as its programmatic dependent
 *   with one CTA per query, selects over the lists (a query's selection
 *   restricted to a range is a prefix of that range's order: Strata PR #3987,
 *   section "Approach").  No CTA waits for another.  `scores` may be NULL; when
 *   given, it also receives the scores (the same values the chained scorer
 *   writes).  `path` must be QSA_PATH_AUTO.  Shapes whose per-CTA scores do not
 *   fit on chip, or whose lists exceed the merge's 4,096 candidates per query
 *   (large k with very long contexts), return QSA_ERR_UNSUPPORTED; use the
 *   chained form for those.
 * Arguments as in qsa_block_scores / qsa_block_topk; ws must hold
 * qsa_workspace_bytes(nq, max_blocks, k, fused) bytes.
 */
qsa_status qsa_select(const void *q, const float *w, const void *kblk, qsa_dtype dt,
                      const int32_t *n_blocks, int nq, int n_heads, int head_dim, int max_blocks,
                      int active_blocks, int k, int32_t *ids, float *scores,
                      int64_t scores_stride, int fused, void *ws, size_t ws_bytes,
                      qsa_path path, qsa_stream stream);

/*
 * Selection attention, forward, over the blocks each query selected: the step
 * that reads the ids, as described in "[wave] NSA: LDS optimization for
 * block-gather in selection attention" (section "Problem": a query reads the
 * tokens of its selected blocks; "LDS staging strategies" 1: the heads of a GQA
 * group read one on-chip copy of each block's K and V).  For query q and
 * attention head h, with KV head g = h / QSA_ATTN_GROUP:
 *
 *   s_t       = dot(qa[q][h][:], K[g][t][:])
 *   o[q][h]   = sum_t exp(scale (s_t - m)) V[g][t][:] / sum_t exp(scale (s_t - m)),  m = max_t s_t
 *   lse[q][h] = scale m + log(sum_t exp(scale (s_t - m)))
 *
 * over the tokens t = 64 b + r (0 <= r < 64) of the distinct ids b >= 0 of
 * ids[q][0..k) with t < n_tokens[q].  A query with no such token gets o = 0 and
 * lse = -inf.
 *
 *   dt        QSA_BF16 or QSA_F16: the format of qa, kcache and vcache_t
 *   qa        [nq][n_heads][128] dtype `dt`, row-major, 16-byte aligned
 *   kcache    [n_kv_heads][capacity][128] dtype `dt` (K[g][t] = token rows), 16-byte aligned
 *   vcache_t  [n_kv_heads][capacity / 64][128][64] dtype `dt`: each 64-token block of V
 *             stored dimension-major, element [g][b][d][r] = V[g][64 b + r][d];
 *             16-byte aligned
 *   ids       [nq][k] int32: block ids (e.g. the ids of qsa_select), -1 = none, in
 *             any order; an id outside [0, ceil(n_tokens[q] / 64)) is skipped and sets
 *             QSA_FLAG_BAD_ID; a repeated id counts once
 *   n_tokens  [nq] int32 on the DEVICE: context length of each query, clamped to
 *             [0, capacity] (a clamp sets QSA_FLAG_NBLOCKS_CLAMPED)
 *   out       [nq][n_heads][128] fp32 out
 *   lse       [nq][n_heads] fp32 out, or NULL
 *   scale     softmax scale (host float), finite and > 0 (usually 1 / sqrt(128))
 *   ws        a workspace of at least 256 bytes (its flags word is used), or NULL
 *             (then device flags are not recorded)
 *
 * Arithmetic: the q.k products on the tensor cores (16-bit x 16-bit -> fp32); the
 * weights exp2((s - m) scale log2 e) in fp32, rounded to `dt` for the P.V product
 * on the tensor cores (-> fp32), and divided by the sum of the rounded weights.
 * Tokens at or past n_tokens take no part, whatever their K and V rows hold.
 * Launch: the kernel is launched as a programmatic dependent of the work before it
 * on `stream`; it reads nothing the caller wrote until that work has completed, so
 * behind a top-k of this library it starts while the top-k finishes.
 * Errors: QSA_ERR_INVALID_ARG for NULL qa/kcache/vcache_t/ids/n_tokens/out,
 * nq < 1, head_dim != 128, n_kv_heads < 1, n_heads != QSA_ATTN_GROUP *
 * n_kv_heads, k outside [1, QSA_ATTN_MAX_K], capacity < 64 or not a multiple of
 * 64, n_kv_heads * capacity >= 2^30, nq * n_heads >= 2^30, misaligned
 * qa/kcache/vcache_t, scale not finite or <= 0, ws smaller than 256 bytes or
 * not 256-byte aligned; QSA_ERR_UNSUPPORTED for a dtype other than QSA_BF16 or
 * QSA_F16.
 */
qsa_status qsa_select_attention(const void *qa, const void *kcache, const void *vcache_t, qsa_dtype dt,
                                const int32_t *ids, int k, const int32_t *n_tokens, int nq, int n_heads,
                                int n_kv_heads, int head_dim, int capacity, float scale, float *out,
                                float *lse, void *ws, size_t ws_bytes, qsa_stream stream);

/*
 * The V cache layout qsa_select_attention reads, from the token-row layout: for
 * every KV head g and every block b in [first_block, first_block + n_blocks),
 * vcache_t[g][b][d][r] = v[g][64 b + r][d] (d < 128, r < 64), copied bit for bit.
 * A cache writer converts the blocks an append touched (the last, partial block
 * again as it fills).  No passage of the source pages defines this call: it
 * serves the layout reading of the attention (each block of V dimension-major, so
 * the P.V product's operand is K-major).
 *
 *   v           [n_kv_heads][capacity][128] 16-bit values (bf16 or fp16), 16-byte aligned
 *   vcache_t    [n_kv_heads][capacity / 64][128][64], same element size, 16-byte aligned;
 *               must not overlap v
 *   capacity    tokens per KV head, a positive multiple of 64
 * Errors: QSA_ERR_INVALID_ARG for NULL or misaligned pointers, n_kv_heads outside
 * [1, 65535], capacity not a positive multiple of 64, n_kv_heads * capacity >= 2^30, a block
 * range outside [0, capacity / 64), n_blocks < 0.
 */
qsa_status qsa_vcache_transpose(const void *v, void *vcache_t, int n_kv_heads, int capacity, int first_block,
                                int n_blocks, qsa_stream stream);

/*
 * ---- The 4-bit KV cache ---------------------------------------------------------
 *
 * K and V rows held in 4 bits per value, for contexts whose 16-bit cache does not fit
 * or whose reading bounds the step (a block is 8,704 bytes per KV head instead of
 * 32,768).  No passage of the source pages defines it: it is this library's form of the
 * reduced KV cache that the pages' engine runs with ("--kv int8"), in the block unit
 * of the selection.
 *
 * Value: each token's row x[0..127] of K (and of V) per KV head has 16 levels,
 *     x ~ scale * code + min,   min = min(x),   scale = least 16-bit number >= (max(x) - min(x)) / 15,
 *     code = (x - min) / scale rounded half to even (0 when scale is 0),
 * so |x - (scale * code + min)| <= scale / 2.  scale and min are held in the rows' own
 * 16-bit format (bf16 or fp16; a minimum of -0 as +0).  A row that holds an infinity or a NaN, or whose range
 * is not finite in fp32, is stored as scale = min = NaN and reads as NaN.
 *
 * Memory: cache [n_kv_heads][capacity / 64][QSA_QCACHE_BLOCK_BYTES], 16-byte aligned, one
 * record per 64-token block:
 *     [   0, 4096)  K codes, 4 planes c of [64 tokens][16 bytes]: byte j of a row holds
 *                   dimension 16c + j (low nibble) and 64 + 16c + j (high nibble)
 *     [4096, 4352)  K pairs [64 tokens]: scale (low 16 bits), min (high 16 bits)
 *     [4352, 4608)  V pairs [64 tokens]
 *     [4608, 8704)  V codes, 2 planes c of [128 dims][16 bytes]: byte j of a row holds
 *                   token 16c + j (low nibble) and 32 + 16c + j (high nibble)
 * Every call on one cache takes the same dt.  Records may be copied as bytes
 * (qsa_gather_blocks).
 */
#define QSA_QCACHE_BLOCK_BYTES 8704

/* Bytes of a cache of these sizes; 0 for invalid ones (n_kv_heads outside [1, 65535],
 * capacity not a positive multiple of 64 or above 64 * QSA_MAX_BLOCKS). */
size_t qsa_qcache_bytes(int n_kv_heads, int capacity);

/*
 * Quantise the K and V rows of n tokens into positions first .. first + n - 1.
 *
 *   k, v        rows of 128 values of dtype `dt` (QSA_BF16 or QSA_F16): token i of KV head g
 *               at k + i * k_token_stride + g * k_head_stride (strides in elements, multiples
 *               of 8, so slices of a fused projection's rows are taken as they lie); 16-byte
 *               aligned
 *   n           tokens, 0 (nothing is enqueued) or more
 *   first       host int, position of the first token; used when first_dev is NULL
 *   first_dev   int32 on the DEVICE, or NULL: the position is read when the call runs (a
 *               captured decode step appends wherever it says).  Tokens whose position lies
 *               outside [0, capacity) are dropped and set QSA_FLAG_NBLOCKS_CLAMPED
 *   cache       see above; other positions, those of a shared byte among them, keep
 *               their values, whatever else writes them meanwhile: appends to different
 *               positions may run at the same time, also in one block
 *   ws          a workspace of at least 256 bytes (its flags word is used), or NULL
 *
 * Errors: QSA_ERR_INVALID_ARG for NULL or misaligned pointers, strides not multiples of 8,
 * head_dim != 128, sizes qsa_qcache_bytes() rejects, n < 0 or > capacity, first < 0 or
 * first + n > capacity (first_dev NULL); QSA_ERR_UNSUPPORTED for another dtype;
 * QSA_ERR_WORKSPACE for a ws smaller than 256 bytes or not 256-byte aligned.
 */
qsa_status qsa_qcache_append(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                             int64_t v_token_stride, int64_t v_head_stride, qsa_dtype dt, int n, int n_kv_heads,
                             int head_dim, int first, const int32_t *first_dev, void *cache, int capacity, void *ws,
                             size_t ws_bytes, qsa_stream stream);

/*
 * The rows of positions first .. first + n - 1 back in 16 bits (scale * code + min rounded once
 * to `dt`; what that puts past dt's largest finite value, by scale / 2 at most, reads as that
 * value), into k and v addressed as for qsa_qcache_append.
 * Errors: as qsa_qcache_append's.
 */
qsa_status qsa_qcache_load(const void *cache, qsa_dtype dt, int n_kv_heads, int head_dim, int capacity, int first,
                           int n, void *k, int64_t k_token_stride, int64_t k_head_stride, void *v,
                           int64_t v_token_stride, int64_t v_head_stride, qsa_stream stream);

/*
 * qsa_select_attention over a 4-bit cache: the same formulas on the rows' values
 * scale * code + min, for n_heads / n_kv_heads = 1 .. 16 query heads per KV head, and each
 * selected block's share of the attention.
 *
 *   qa        query i, head h at qa + i * q_stride + h * q_head_stride, 128 values of dtype
 *             `dt` (strides in elements, multiples of 8), 16-byte aligned
 *   cache     of the same dt
 *   ids, k, n_tokens, capacity, scale, ws   as for qsa_select_attention
 *   out       [nq][n_heads][128] of dtype out_dt: QSA_F32, or dt (what passes dt's range becomes
 *             its largest finite value)
 *   lse       [nq][n_heads] fp32 out, or NULL
 *   weights   [nq][n_kv_heads][k] fp32 out, or NULL: the softmax weight that the group's heads
 *             together give to slot j's tokens (a slot with id -1, an id outside the
 *             context, or a repeat of an earlier slot gets 0); a (query, KV head)'s
 *             weights add up to its heads, or to 0 when it sees no token
 *
 * Arithmetic: products of codes with the queries exact (queries to 2^-18 of their head's
 * largest value), accumulated in fp32; softmax statistics, lse and weights in fp32; the
 * weights of the P.V product are rounded to 8 significant bits beside bf16 rows and 12 beside
 * fp16 ones, and to 2^-18 of the largest weight times the largest V scale where they are
 * smaller.  Sums over the tokens are formed in fp32 before they are divided by the weights' sum:
 * bf16 rows of V above 2^80 in magnitude may overflow.
 * Launch: as a programmatic dependent of the work before it on `stream`, as
 * qsa_select_attention.
 * Errors: as qsa_select_attention's, with n_heads a multiple of n_kv_heads of at most 16
 * times it, the cache sizes as qsa_qcache_bytes() has them, nq * n_kv_heads < 2^28, and
 * out_dt other than QSA_F32 or dt.
 */
qsa_status qsa_select_attention_qcache(const void *qa, int64_t q_stride, int64_t q_head_stride, qsa_dtype dt,
                                       const void *cache, const int32_t *ids, int k, const int32_t *n_tokens, int nq,
                                       int n_heads, int n_kv_heads, int head_dim, int capacity, float scale, void *out,
                                       qsa_dtype out_dt, float *lse, float *weights, void *ws, size_t ws_bytes,
                                       qsa_stream stream);

/*
 * ---- Eviction by accumulated attention weight ------------------------------------
 *
 * Blocks that the attention no longer looks at leave the cache: the weights of each
 * attention call are added up per block (qsa_block_weights_add, with a decay), the blocks
 * to keep are those of largest sum beside the first and the most recent ones
 * (qsa_evict_plan), and their records, in every array that holds one record per block,
 * move together in order (qsa_gather_blocks).  No passage of the source pages defines these
 * calls; "block" is the selection's 64-token block, so the indexer's keys move along.
 */

/* Largest weight qsa_block_weights_add takes (an attention call's are at most 16). */
#define QSA_MAX_BLOCK_WEIGHT 32.0f

/*
 * acc[b] = decay * prev[b] + the sum of weights[q][g][j] over all q, g, j with ids[q][j] == b.
 *
 *   weights   [nq][n_kv_heads][k] fp32 in [0, QSA_MAX_BLOCK_WEIGHT] (others are clamped, NaN to 0,
 *             and set QSA_FLAG_BAD_WEIGHT)
 *   ids       [nq][k] int32; -1 is skipped, other ids outside [0, max_blocks) too (with
 *             QSA_FLAG_BAD_ID); the same id may appear any number of times
 *   decay     host double, finite and >= 0; the product with prev and the sum are formed in 64 bits
 *             and rounded to fp32 once
 *   prev      [max_blocks] fp32, or NULL (zeros); may be acc itself
 *   acc       [max_blocks] fp32 out
 *   ws        a workspace of at least 256 bytes (its flags word is used), or NULL
 *
 * The weights are summed as integers in units of 2^-36, so the result does not depend on
 * the order of the work.
 * Errors: QSA_ERR_INVALID_ARG for NULL pointers, nq, n_kv_heads or k < 1, nq * n_kv_heads * k >
 * 2^22, max_blocks outside [1, QSA_MAX_BLOCKS], a decay not finite or < 0, a prev that
 * overlaps acc without being it, weights or ids that overlap acc; QSA_ERR_WORKSPACE as above.
 */
qsa_status qsa_block_weights_add(const float *weights, const int32_t *ids, int nq, int n_kv_heads, int k, double decay,
                                 const float *prev, float *acc, int max_blocks, void *ws, size_t ws_bytes,
                                 qsa_stream stream);

/*
 * Which blocks stay, for each of n_rows caches (rows): of a row's nb = ceil(n_tokens / 64)
 * blocks the first n_first, the last n_last, and of the others those of largest weight (ties
 * to the lower id), n_keep in all; all of them when nb <= n_keep.
 *
 *   weights     [n_rows][weights_stride] fp32, weights_stride >= max_blocks (a NaN ranks below
 *               every number)
 *   n_tokens    [n_rows] int32 on the DEVICE, clamped to [0, 64 * max_blocks] (a clamp sets
 *               QSA_FLAG_NBLOCKS_CLAMPED)
 *   keep        [n_rows][n_keep] int32 out: the kept ids in ascending order, -1 behind them
 *   new_tokens  [n_rows] int32 out: tokens left, n_tokens - 64 * (blocks evicted): the last
 *               block stays last, so a partial one stays valid.  May be n_tokens itself (lengths
 *               updated in place); otherwise keep and new_tokens overlap nothing
 *   ws          a workspace of at least 256 bytes (its flags word is used), or NULL
 *
 * Launch: as a programmatic dependent of the work before it, and a qsa_gather_blocks behind it
 * may line up while it runs (both wait before they read anything).
 * Errors: QSA_ERR_INVALID_ARG for NULL pointers, n_rows outside [1, 2^20], max_blocks outside
 * [1, QSA_MAX_BLOCKS], weights_stride < max_blocks, n_keep outside [1, max_blocks],
 * n_first < 0, n_last < 1, n_first + n_last > n_keep, an output that overlaps an input or the
 * other output (but for new_tokens == n_tokens); QSA_ERR_WORKSPACE as above.
 */
qsa_status qsa_evict_plan(const float *weights, int64_t weights_stride, const int32_t *n_tokens, int n_rows,
                          int max_blocks, int n_keep, int n_first, int n_last, int32_t *keep, int32_t *new_tokens,
                          void *ws, size_t ws_bytes, qsa_stream stream);

/* An array that holds one record of block_bytes per block: src [n_rows][src_blocks] records,
 * dst [n_rows][dst_blocks] (a row per KV head for a cache, one row for the indexer's keys). */
typedef struct {
    const void *src;
    void *dst;
    int64_t block_bytes; /* a multiple of 4 */
    int32_t n_rows;
    int32_t src_blocks;
    int32_t dst_blocks;
} qsa_block_array;

#define QSA_GATHER_MAX_ARRAYS 8

/*
 * dst[row][i] = src[row][keep[i]] for 0 <= i < n_keep, for each of n_arrays (host array, 1 ..
 * QSA_GATHER_MAX_ARRAYS) arrays, one launch in all.
 *
 *   keep   [n_keep] int32 on the DEVICE (a row of qsa_evict_plan's): where it is -1, or outside
 *          [0, src_blocks) (QSA_FLAG_BAD_ID), dst[row][i] is left as it was
 *   ws     a workspace of at least 256 bytes (its flags word is used), or NULL
 *
 * Out of place: a dst may overlap no src, no other dst and not keep.
 * Errors: QSA_ERR_INVALID_ARG for NULL pointers, n_arrays or n_keep out of range, sizes < 1,
 * dst_blocks < n_keep, block_bytes not a multiple of 4 or above 2^30, pointers not 4-byte
 * aligned, a dst that overlaps; QSA_ERR_WORKSPACE as above.
 */
qsa_status qsa_gather_blocks(const qsa_block_array *arrays, int n_arrays, const int32_t *keep, int n_keep, void *ws,
                             size_t ws_bytes, qsa_stream stream);

/*
 * Copy the workspace flags word (QSA_FLAG_* bits) to host `*flags`, waiting for
 * `stream` to finish; clear it on the device when `clear` is nonzero.
 */
qsa_status qsa_read_flags(void *ws, uint32_t *flags /* host */, int clear, qsa_stream stream);

/* The path QSA_PATH_AUTO takes for these host-visible sizes (no launch). */
qsa_path qsa_auto_path(int nq, int max_blocks, int active_blocks, int k);

/* One-line reason for the last error status returned on this thread. */
const char *qsa_last_error(void);

/* QSA_VERSION of the loaded library. */
int qsa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QSA_H */
