// pages.cu -- the pages of a 16-bit cache shared by many sequences: fork, release, reserve, compact and append
// (the copy of whole pages is gather_blocks_kernel's).
//
// What a page's entry in a table says is in qsa.h.  The bookkeeping reads and writes a few KB, so its time is a launch
// and a chain of loads; what there is to choose is the number of steps in that chain.
//  - fork, release: one CTA per row, references by atomics (integers: any order gives the same).
//  - reserve: one CTA.  A thread, a warp or the whole CTA counts what a row lacks, by the entries it looks at; shared last
//    pages are settled by rank among the rows that write (a row copies when more references than rows before it
//    remain); one scan gives each row its part of the ascending list of free pages, from which its entries are filled.
//    The list is written no further than it is needed.
//  - compact: one CTA lists the free pages below the number of live ones and the live pages behind it, both in order,
//    and pairs them; a second grid rewrites the table.
//  - append: a CTA looks a page up and takes some or all of its KV heads: K rows as they are, V through shared memory into its
//    dimension-major block.  Bound by HBM where rows are long: each is read once and written once; where they are many and short,
//    by the rows before its own that every CTA sums up (4,000 rows of a token, 8 heads, 132 us, with ends 139).
// Measured: reserve and append for 8 sequences of up to 16 rows 11 us; for one of 131,072 rows, 4 KV heads, 97 us (537 MB, 5.5
// TB/s; V transposed by words, by 16-bit elements 145); release, fork, reserve and the copied last pages for 8 sequences
// forked into 64 14 us; the moves of 4,096 pages (4 KV heads, 55 % live) worked out and copied 52.5 us (of which 39 for the bytes).
#include <cstdint>

#include "launch.h"
#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int kRowThreads = 256;    // fork, release, append
constexpr int kOneThreads = 1024;   // reserve, compact
constexpr int kBatch = 4;           // table entries of a thread under way (1: 2,049 of them 2 us more)
// reserve: entries of a row that one thread looks at, that a warp does (a row each), and beyond them the whole CTA (row by row).  Us:
constexpr int kFew = 2;             // 8 rows with up to 2 each 10.9, by warps 11.8; 8 a thread: 64 rows with 6 each 17.9 against 20, 8 with 2 11.1
constexpr int kMany = 128;          // one row with 313: 20.4, by a warp 23.4; 8 rows with 47 by warps 17.7, by the CTA 26.4

__device__ __forceinline__ void raise(uint32_t *flags, uint32_t bit) {
    if (flags) atomicOr(flags, bit);
}
// A length clamped to what a row can hold.
__device__ __forceinline__ int row_tokens(int n, int max_pages, uint32_t *flags) {
    const int most = max_pages * 64;
    if (n < 0 || n > most) {
        raise(flags, QSA_FLAG_NBLOCKS_CLAMPED);
        return n < 0 ? 0 : most;
    }
    return n;
}
// A page that nothing referred to when a reference was given back: as before.
__device__ __forceinline__ void restore(int32_t *refs, int page, uint32_t *flags) {
    atomicAdd(refs + page, 1);
    raise(flags, QSA_FLAG_BAD_ID);
}

__global__ void __launch_bounds__(kRowThreads) pages_fork_kernel(PageTable t, int32_t *n_tokens, int32_t *refs,
                                                                 const int32_t *src, const int32_t *dst, int n) {
    wait_prior_grid();
    allow_dependent_launch();
    const int i = blockIdx.x, tid = threadIdx.x, from = src[i], to = dst[i];
    if (from == -1 && to == -1) return;
    bool bad = from < 0 || from >= t.n_rows || to < 0 || to >= t.n_rows;
    for (int j = tid; j < n; j += kRowThreads) bad = bad || src[j] == to || (j < i && dst[j] == to);
    bad = __syncthreads_or(bad);
    // only one entry of the call reads and writes row `to` from here on, and none reads it as a source
    if (!bad) bad = n_tokens[to] > 0;
    if (bad) {
        if (tid == 0) raise(t.flags, QSA_FLAG_BAD_ID);
        return;
    }
    const int tokens = row_tokens(n_tokens[from], t.max_pages, t.flags), nb = (tokens + 63) >> 6;
    const int32_t *a = t.table + (size_t)from * t.stride;
    int32_t *b = t.table + (size_t)to * t.stride;
    for (int j = tid; j < t.max_pages; j += kRowThreads) {
        const int had = b[j];
        int page = j < nb ? a[j] : -1;
        if (j < nb && (page < 0 || page >= t.n_pages)) {
            raise(t.flags, QSA_FLAG_BAD_ID);
            page = -1;
        }
        if (page >= 0) atomicAdd(refs + page, 1);
        if (had >= 0 && had < t.n_pages && atomicSub(refs + had, 1) <= 0) restore(refs, had, t.flags);
        if (had != page) b[j] = page;
    }
    __syncthreads();   // every thread has read n_tokens[to]
    if (tid == 0) n_tokens[to] = tokens;
}

__global__ void __launch_bounds__(kRowThreads) pages_release_kernel(PageTable t, int32_t *n_tokens, int32_t *refs,
                                                                    const int32_t *keep) {
    wait_prior_grid();
    allow_dependent_launch();
    const int row = blockIdx.x, tid = threadIdx.x, left = keep[row], n = n_tokens[row];
    if (left < 0) return;
    int32_t *a = t.table + (size_t)row * t.stride;
    for (int j0 = (int)(((unsigned)left + 63u) >> 6) + tid; j0 < t.max_pages; j0 += kBatch * kRowThreads) {
        int page[kBatch], held[kBatch];   // loads and atomics of a batch under way together
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = j0 + i * kRowThreads;
            page[i] = j < t.max_pages ? a[j] : -1;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            held[i] = page[i] >= 0 && page[i] < t.n_pages ? atomicSub(refs + page[i], 1) : 1;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (page[i] == -1) continue;
            if (page[i] < 0 || page[i] >= t.n_pages) {
                raise(t.flags, QSA_FLAG_BAD_ID);
                continue;
            }
            if (held[i] <= 0) restore(refs, page[i], t.flags);
            a[j0 + i * kRowThreads] = -1;
        }
    }
    __syncthreads();   // keep may be n_tokens: every thread has read it
    if (tid == 0 && left < n) n_tokens[row] = left;
}

// Inclusive scan of one value per thread over the CTA's 1,024 threads; total in `total`.
__device__ __forceinline__ unsigned long long scan_all(unsigned long long v, unsigned long long *sums,
                                                       unsigned long long &total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const unsigned long long x = __shfl_up_sync(~0u, v, d);
        if (lane >= d) v += x;
    }
    __syncthreads();   // earlier readers of sums
    if (lane == 31) sums[wid] = v;
    __syncthreads();
    unsigned long long before = 0ull;
    total = 0ull;
#pragma unroll 8
    for (int w = 0; w < kOneThreads / 32; ++w) {
        if (w < wid) before += sums[w];
        total += sums[w];
    }
    return before + v;
}

// What a row of reserve does with its last page.
// (kPast: the row is refused for where its tokens would go, past its entries or in a page that others refer to.)
enum : uint8_t { kWhole = 0, kCopies = 1, kKeeps = 2, kPast = 3 };

// The entries that a row's new tokens need, [b0, b1), and whether it has any.
struct Wants {
    int n, more, b0, b1;
    bool past;
};
__device__ __forceinline__ Wants wants_of(const PageTable &t, const int32_t *n_tokens, const int32_t *add, int row, bool tell) {
    Wants w;
    w.n = n_tokens[row];
    w.more = add[row];
    if (w.more < 0) {
        if (tell) raise(t.flags, QSA_FLAG_NBLOCKS_CLAMPED);
        w.more = 0;
    }
    w.past = w.n < 0 || (long long)w.n + w.more > 64ll * t.max_pages;
    w.b0 = w.b1 = 0;
    if (!w.past && w.more > 0) {
        w.b0 = (w.n + 63) >> 6;
        w.b1 = (int)(((long long)w.n + w.more + 63) >> 6);
    }
    return w;
}
__device__ __forceinline__ bool is_page(const PageTable &t, int p) { return p >= 0 && p < t.n_pages; }

__global__ void __launch_bounds__(kOneThreads) pages_reserve_kernel(PageTable t, const int32_t *n_tokens, int32_t *refs,
                                                                    const int32_t *add, int32_t *new_tokens,
                                                                    int32_t *copy_src, int32_t *copy_dst, PagesWs ws) {
    __shared__ int32_t last[QSA_MAX_TABLE_ROWS];   // the page a row is about to write into, or -1
    __shared__ int32_t needs[QSA_MAX_TABLE_ROWS];  // pages it asks for
    __shared__ uint8_t what[QSA_MAX_TABLE_ROWS];
    __shared__ unsigned long long sums[kOneThreads / 32];
    __shared__ int counts[kOneThreads / 32];
    wait_prior_grid();
    allow_dependent_launch();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    int held[4];   // references of the pool's first pages, on their way meanwhile
#pragma unroll
    for (int e = 0; e < 4; ++e) held[e] = tid * 4 + e < t.n_pages ? refs[tid * 4 + e] : 1;
    // what each row lacks: entries that are no page (a bad one counts as none).  A page behind its tokens that others refer to
    // as well may hold theirs: the row is refused.  (Rows in step with their pages have none there, and nothing is loaded.)
    bool any_warp = false, any_all = false;
    for (int row = tid; row < t.n_rows; row += kOneThreads) {
        const Wants w = wants_of(t, n_tokens, add, row, true);
        const int32_t *a = t.table + (size_t)row * t.stride;
        int lacks = 0, page = -1;
        bool others = false;
        if (w.past) raise(t.flags, QSA_FLAG_NBLOCKS_CLAMPED);
        if (w.b1 - w.b0 <= kFew) {
            int p[kFew];
#pragma unroll
            for (int i = 0; i < kFew; ++i) p[i] = w.b0 + i < w.b1 ? a[w.b0 + i] : 0;
            if (w.b1 > 0 && (w.n & 63)) page = a[w.n >> 6];
#pragma unroll
            for (int i = 0; i < kFew; ++i) {
                lacks += w.b0 + i < w.b1 && !is_page(t, p[i]);
                if (p[i] < -1 || p[i] >= t.n_pages) raise(t.flags, QSA_FLAG_BAD_ID);
                others = others || (w.b0 + i < w.b1 && is_page(t, p[i]) && refs[p[i]] > 1);
            }
        } else {
            if (w.n & 63) page = a[w.n >> 6];
            any_warp = any_warp || w.b1 - w.b0 <= kMany;
            any_all = any_all || w.b1 - w.b0 > kMany;
        }
        if (w.b1 > 0 && (w.n & 63) && !is_page(t, page)) {   // a page that the tokens should have lain in
            raise(t.flags, QSA_FLAG_BAD_ID);
            page = -1;
            ++lacks;
        }
        if (others) raise(t.flags, QSA_FLAG_BAD_ID);
        last[row] = others ? -1 : page;
        what[row] = w.past || others ? kPast : kWhole;
        needs[row] = lacks;
    }
    if (__syncthreads_or(any_warp))
        for (int row = wid; row < t.n_rows; row += kOneThreads / 32) {
            const Wants w = wants_of(t, n_tokens, add, row, false);
            if (w.b1 - w.b0 <= kFew || w.b1 - w.b0 > kMany) continue;
            const int32_t *a = t.table + (size_t)row * t.stride;
            int lacks = 0;
            bool others = false;
#pragma unroll 4
            for (int b = w.b0 + lane; b < w.b1; b += 32) {
                const int p = a[b];
                lacks += !is_page(t, p);
                if (p < -1 || p >= t.n_pages) raise(t.flags, QSA_FLAG_BAD_ID);
                others = others || (is_page(t, p) && refs[p] > 1);
            }
            lacks = __reduce_add_sync(~0u, lacks);
            others = __any_sync(~0u, others);
            if (lane == 0) {
                needs[row] += lacks;
                if (others) {
                    raise(t.flags, QSA_FLAG_BAD_ID);
                    last[row] = -1;
                    what[row] = kPast;
                }
            }
        }
    if (__syncthreads_or(any_all))
        for (int row = 0; row < t.n_rows; ++row) {
            const Wants w = wants_of(t, n_tokens, add, row, false);
            if (w.b1 - w.b0 <= kMany) continue;
            const int32_t *a = t.table + (size_t)row * t.stride;
            int lacks = 0;
            bool others = false;
#pragma unroll 4
            for (int b = w.b0 + tid; b < w.b1; b += kOneThreads) {
                const int p = a[b];
                lacks += !is_page(t, p);
                if (p < -1 || p >= t.n_pages) raise(t.flags, QSA_FLAG_BAD_ID);
                others = others || (is_page(t, p) && refs[p] > 1);
            }
            lacks = __reduce_add_sync(~0u, lacks);
            if (lane == 0) atomicAdd(&needs[row], lacks);
            if (others) {   // the same by every thread that says so
                raise(t.flags, QSA_FLAG_BAD_ID);
                last[row] = -1;
                what[row] = kPast;
            }
        }
    __syncthreads();
    // rows that share their last page: the k-th of them to write copies while more than k references remain
    for (int row = tid; row < t.n_rows; row += kOneThreads) {
        const int page = last[row];
        if (what[row] == kPast) needs[row] = 0;   // asks for none
        if (page < 0) continue;
        const int all = refs[page];
        if (all <= 1) continue;
        int earlier = 0;
        for (int j = 0; j < row; ++j) earlier += last[j] == page;
        const bool copies = all - earlier > 1;
        what[row] = copies ? kCopies : kKeeps;
        if (copies) needs[row] += 1;
    }
    __syncthreads();
    // pages that a row and those before it ask for
    unsigned long long asked = 0ull;
    for (int r0 = 0; r0 < t.n_rows; r0 += kOneThreads) {
        const int row = r0 + tid;
        unsigned long long total;
        const unsigned long long incl = scan_all(row < t.n_rows ? (unsigned long long)needs[row] : 0ull, sums, total);
        if (row < t.n_rows) {   // more than a pool holds is more than is free
            const unsigned long long upto = asked + incl;
            ws.upto[row] = (int)(upto < (1ull << 30) ? upto : (1ull << 30));
        }
        asked += total;
    }
    const int want = (int)(asked < (unsigned long long)t.n_pages ? asked : (unsigned long long)t.n_pages);
    // the first free pages in order, as many as are asked for
    int free_pages = 0;
    for (int p0 = 0; p0 < t.n_pages && free_pages < want; p0 += 4 * kOneThreads) {
        int k = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = p0 + tid * 4 + e;
            if (p0 > 0) held[e] = p < t.n_pages ? refs[p] : 1;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) k += held[e] == 0;
        const int incl = warp_incl_scan(k);
        __syncthreads();
        if (lane == 31) counts[wid] = incl;
        __syncthreads();
        int at = free_pages + incl - k;
        for (int w = 0; w < kOneThreads / 32; ++w) {
            const int c = counts[w];
            if (w < wid) at += c;
            free_pages += c;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (held[e] == 0) {
                if (at < want) ws.list[at] = p0 + tid * 4 + e;
                ++at;
            }
    }
    __syncthreads();   // the list and the rows' needs lie in global memory, read by other threads of this CTA
    // the page under a row's last tokens comes first, then the others; a row's first page for them
    auto served = [&](int row, int &need) {
        need = needs[row];
        const uint8_t does = what[row];
        return does != kPast && (ws.upto[row] <= free_pages || (need == 0 && does != kKeeps));
    };
    auto first_of = [&](int row, int need, const Wants &w) {
        return ws.upto[row] - need + ((w.n & 63) && (what[row] == kCopies || last[row] < 0) ? 1 : 0);
    };
    for (int row = tid; row < t.n_rows; row += kOneThreads) {
        const Wants w = wants_of(t, n_tokens, add, row, false);
        int need, from = -1, to = -1;
        const bool ok = served(row, need);
        if (ok && need > 0) {
            int32_t *a = t.table + (size_t)row * t.stride;
            int at = first_of(row, need, w);
            if (at > ws.upto[row] - need) {
                to = ws.list[at - 1];
                a[w.n >> 6] = to;
                refs[to] = 1;
                if (what[row] == kCopies) {
                    from = last[row];
                    atomicSub(refs + from, 1);
                } else {
                    to = -1;   // nothing to copy
                }
            }
            if (w.b1 - w.b0 <= kFew)
#pragma unroll
                for (int i = 0; i < kFew; ++i)
                    if (w.b0 + i < w.b1 && !is_page(t, a[w.b0 + i])) {
                        const int page = ws.list[at++];
                        a[w.b0 + i] = page;
                        refs[page] = 1;
                    }
        }
        if (!ok && what[row] != kPast) raise(t.flags, QSA_FLAG_NO_PAGES);
        new_tokens[row] = ok ? w.n + w.more : w.n;
        copy_src[row] = from;
        copy_dst[row] = to;
    }
    if (__syncthreads_or(any_warp))
        for (int row = wid; row < t.n_rows; row += kOneThreads / 32) {
            const Wants w = wants_of(t, n_tokens, add, row, false);
            int need;
            if (w.b1 - w.b0 <= kFew || w.b1 - w.b0 > kMany || !served(row, need) || need == 0) continue;
            int32_t *a = t.table + (size_t)row * t.stride;
            int at = first_of(row, need, w);
            for (int b = w.b0; b < w.b1; b += 32) {
                const bool lacks = b + lane < w.b1 && !is_page(t, a[b + lane]);
                const unsigned who = __ballot_sync(~0u, lacks);
                if (lacks) {
                    const int page = ws.list[at + __popc(who & ((1u << lane) - 1u))];
                    a[b + lane] = page;
                    refs[page] = 1;
                }
                at += __popc(who);
            }
        }
    if (__syncthreads_or(any_all))
        for (int row = 0; row < t.n_rows; ++row) {
            const Wants w = wants_of(t, n_tokens, add, row, false);
            int need;
            if (w.b1 - w.b0 <= kMany || !served(row, need) || need == 0) continue;
            int32_t *a = t.table + (size_t)row * t.stride;
            int at = first_of(row, need, w);
            for (int b = w.b0; b < w.b1; b += kOneThreads) {
                const bool lacks = b + tid < w.b1 && !is_page(t, a[b + tid]);
                unsigned long long total;
                const int rank = (int)scan_all(lacks ? 1ull : 0ull, sums, total) - 1;
                if (lacks) {
                    const int page = ws.list[at + rank];
                    a[b + tid] = page;
                    refs[page] = 1;
                }
                at += (int)total;
            }
        }
}

__global__ void __launch_bounds__(kOneThreads) pages_compact_kernel(const int32_t *refs, int n_pages, int32_t *refs_out,
                                                                    int32_t *copy_src, int32_t *copy_dst, PagesWs ws) {
    __shared__ int counts[2][kOneThreads / 32];
    wait_prior_grid();
    allow_dependent_launch();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    int mine = 0;
#pragma unroll 4
    for (int p = tid; p < n_pages; p += kOneThreads) mine += refs[p] > 0;
    mine = __reduce_add_sync(~0u, mine);
    if (lane == 0) counts[0][wid] = mine;
    __syncthreads();
    int live = 0;
    for (int w = 0; w < kOneThreads / 32; ++w) live += counts[0][w];
    // free pages in front of `live` and live ones behind, each in order
    int holes = 0, moves = 0;
    for (int p0 = 0; p0 < n_pages; p0 += 4 * kOneThreads) {
        bool hole[4], moved[4];
        int kh = 0, km = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = p0 + tid * 4 + e;
            const bool is_live = p < n_pages && refs[p] > 0;
            hole[e] = p < live && !is_live;
            moved[e] = p >= live && is_live;
            kh += hole[e];
            km += moved[e];
        }
        const int ih = warp_incl_scan(kh), im = warp_incl_scan(km);
        __syncthreads();
        if (lane == 31) {
            counts[0][wid] = ih;
            counts[1][wid] = im;
        }
        __syncthreads();
        int ah = holes + ih - kh, am = moves + im - km;
        for (int w = 0; w < kOneThreads / 32; ++w) {
            const int ch = counts[0][w], cm = counts[1][w];
            if (w < wid) {
                ah += ch;
                am += cm;
            }
            holes += ch;
            moves += cm;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = p0 + tid * 4 + e;
            if (hole[e]) copy_dst[ah++] = p;
            if (moved[e]) copy_src[am++] = p;
            else if (p >= live && p < n_pages) ws.list[p] = -1;   // a table entry that names it names nothing
        }
    }
    __syncthreads();   // holes == moves
    for (int i = tid; i < moves; i += kOneThreads) {
        const int from = copy_src[i], to = copy_dst[i], r = refs[from];
        ws.list[from] = to;
        refs_out[to] = r;
        refs_out[from] = 0;
    }
    for (int i = moves + tid; i < n_pages / 2; i += kOneThreads) copy_src[i] = copy_dst[i] = -1;
    // what stays: refs of moved pages and of the holes are not looked at again when refs_out is refs
    if (refs_out != refs)
        for (int p = tid; p < n_pages; p += kOneThreads) {
            const int r = refs[p];
            if (p < live ? r > 0 : r <= 0) refs_out[p] = p < live ? r : 0;
        }
    if (tid == 0) *ws.live = live;
}

__global__ void __launch_bounds__(kRowThreads) pages_retable_kernel(PageTable t, int32_t *table_out, PagesWs ws) {
    wait_prior_grid();
    allow_dependent_launch();
    const int live = *ws.live;
    const long long all = (long long)t.n_rows * t.max_pages;
    for (long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x; i < all; i += (long long)gridDim.x * kRowThreads) {
        const int row = (int)(i / t.max_pages), j = (int)(i - (long long)row * t.max_pages);
        const size_t at = (size_t)row * t.stride + j;
        const int page = t.table[at];
        int to = -1;
        if (page >= 0 && page < live) to = page;
        else if (page >= live && page < t.n_pages) to = ws.list[page];
        if (to < 0 && page != -1) raise(t.flags, QSA_FLAG_BAD_ID);
        table_out[at] = to;
    }
}

// What a CTA of the append writes: the index-th page that a row's entries touch; row < 0: nothing.
struct Unit {
    int row, index;
};
// The entries of a row, and where they go.
struct Span {
    int e0;            // first entry
    long long lo, hi;  // positions
    int first;
    bool falls;        // cu_rows descends here
};
__device__ __forceinline__ Span span_of(const PageTable &t, const PagesAppendArgs &a, int row, bool tell) {
    Span s;
    int c0 = a.cu_rows[row], c1 = a.cu_rows[row + 1];
    if (tell && (c0 < 0 || c0 > a.n || c1 < c0 || c1 > a.n)) raise(t.flags, QSA_FLAG_NBLOCKS_CLAMPED);
    s.falls = c1 < c0;
    c0 = min(max(c0, 0), a.n);
    c1 = min(max(c1, c0), a.n);
    s.e0 = c0;
    s.first = a.first[row];
    const long long end = (long long)s.first + (c1 - c0), most = 64ll * t.max_pages;
    s.lo = s.first < 0 ? 0 : s.first;
    s.hi = end > most ? most : end;
    if (tell && c1 > c0 && (s.first < 0 || end > most)) raise(t.flags, QSA_FLAG_NBLOCKS_CLAMPED);
    if (a.end) s.hi = min(s.hi, (long long)a.end[row]);   // where the row's room ends
    if (s.hi < s.lo || c1 == c0) s.hi = s.lo;
    return s;
}
__device__ __forceinline__ int pages_of(const Span &s) { return s.hi > s.lo ? (int)(((s.hi + 63) >> 6) - (s.lo >> 6)) : 0; }

__global__ void __launch_bounds__(kRowThreads) pages_append_kernel(PageTable t, PagesAppendArgs a) {
    __shared__ BlockScratch sm;
    __shared__ Unit unit;
    // V rows of a page, 16 units of 16 bytes each: unit u of token i lies at u ^ (i / 8), so that neither the rows coming in
    // nor eight tokens of a dimension going out meet a bank twice
    __shared__ uint4 tile[64][16];
    __shared__ int source[64];
    __shared__ int fall;   // the first row at which cu_rows descends, of those looked at
    wait_prior_grid();
    allow_dependent_launch();
    const int tid = threadIdx.x;
    if (tid == 0) {
        unit.row = -1;
        fall = t.n_rows;
    }
    __syncthreads();
    const bool tell = blockIdx.x == gridDim.x - 1 && blockIdx.y == 0;   // looks at every row
    int before = 0;
    for (int r0 = 0; r0 < t.n_rows && (tell || before <= (int)blockIdx.x); r0 += kRowThreads) {
        const int row = r0 + tid;
        int np = 0, total;
        if (row < t.n_rows) {
            const Span s = span_of(t, a, row, tell);
            np = pages_of(s);
            if (s.falls) atomicMin(&fall, row);
        }
        const int at = before + block_excl_scan<kRowThreads>(np, sm, total);
        if ((int)blockIdx.x >= at && (int)blockIdx.x < at + np) {
            unit.row = row;
            unit.index = (int)blockIdx.x - at;
        }
        if (before <= (int)blockIdx.x) before += total;   // up to 2^28 pages a turn; in all they may be more than an int holds
    }
    __syncthreads();
    // Rows up to a descent hold n entries at most, and the grid has a CTA for each of their pages.  Those behind it could
    // hold the same ones over again: they take none.
    const int row = unit.row;
    if (row < 0 || row > fall) return;
    const Span s = span_of(t, a, row, false);
    const int b = (int)(s.lo >> 6) + unit.index;
    const int page = t.table[(size_t)row * t.stride + b];
    if (page < 0 || page >= t.n_pages) {
        if (tid == 0) raise(t.flags, QSA_FLAG_BAD_ID);
        return;
    }
    if (tid < 64) {   // the row that each of the page's tokens comes from
        const long long pos = (long long)b * 64 + tid;
        int r = -1;
        if (pos >= s.lo && pos < s.hi) {
            const int e = s.e0 + (int)(pos - s.first);
            r = a.rows ? a.rows[e] : e;
            if (r < 0 || r >= a.n_source) {
                if (r != -1 && blockIdx.y == 0) raise(t.flags, QSA_FLAG_BAD_ID);
                r = -1;
            }
        }
        source[tid] = r;
    }
    __syncthreads();
    const int u = tid & 15, c = tid & 7;
    uint32_t there = 0u;   // of the eight tokens that this thread writes
#pragma unroll
    for (int j = 0; j < 8; ++j) there |= (source[8 * c + j] >= 0 ? 1u : 0u) << j;
    for (int g = blockIdx.y; g < a.n_kv_heads; g += gridDim.y) {
        const uint16_t *k = static_cast<const uint16_t *>(a.k.p) + (size_t)g * a.k.head;
        const uint16_t *v = static_cast<const uint16_t *>(a.v.p) + (size_t)g * a.v.head;
        uint16_t *kc = static_cast<uint16_t *>(a.kcache) + ((size_t)g * t.n_pages + page) * (64 * 128);
        uint16_t *vc = static_cast<uint16_t *>(a.vcache_t) + ((size_t)g * t.n_pages + page) * (64 * 128);
        uint4 kx[4], vx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = source[(tid >> 4) + 16 * i];
            kx[i] = vx[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r >= 0) {
                kx[i] = *reinterpret_cast<const uint4 *>(k + (int64_t)r * a.k.token + 8 * u);
                vx[i] = *reinterpret_cast<const uint4 *>(v + (int64_t)r * a.v.token + 8 * u);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = (tid >> 4) + 16 * i;
            if (source[at] >= 0) *reinterpret_cast<uint4 *>(kc + at * 128 + 8 * u) = kx[i];
            tile[at][u ^ (at >> 3)] = vx[i];
        }
        __syncthreads();
        // two dimensions and eight tokens a turn; 8 lanes write a dimension's 128 bytes
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int pair = (tid >> 3) + 32 * i;   // dimensions 2 pair and 2 pair + 1
            uint32_t x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = reinterpret_cast<const uint32_t *>(&tile[8 * c + j][(pair >> 2) ^ c])[pair & 3];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint16_t *to = vc + (2 * pair + h) * 64 + 8 * c;
                const uint32_t pick = h ? 0x7632u : 0x5410u;   // a half of two words
                if (there == 0xFFu) {
                    *reinterpret_cast<uint4 *>(to) = make_uint4(__byte_perm(x[0], x[1], pick), __byte_perm(x[2], x[3], pick),
                                                                __byte_perm(x[4], x[5], pick), __byte_perm(x[6], x[7], pick));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (there >> j & 1u) to[j] = (uint16_t)(h ? x[j] >> 16 : x[j]);
                }
            }
        }
        __syncthreads();
    }
}

}  // namespace

qsa_status launch_pages_fork(const PageTable &t, int32_t *n_tokens, int32_t *refs, const int32_t *src, const int32_t *dst,
                             int n, cudaStream_t s) {
    return launch_dependent("pages_fork_kernel launch", pages_fork_kernel, n, kRowThreads, 0, s, t, n_tokens, refs, src, dst, n);
}
qsa_status launch_pages_release(const PageTable &t, int32_t *n_tokens, int32_t *refs, const int32_t *keep, cudaStream_t s) {
    return launch_dependent("pages_release_kernel launch", pages_release_kernel, t.n_rows, kRowThreads, 0, s, t, n_tokens, refs,
                            keep);
}
qsa_status launch_pages_reserve(const PageTable &t, const int32_t *n_tokens, int32_t *refs, const int32_t *add,
                                int32_t *new_tokens, int32_t *copy_src, int32_t *copy_dst, const PagesWs &ws,
                                cudaStream_t s) {
    return launch_dependent("pages_reserve_kernel launch", pages_reserve_kernel, 1, kOneThreads, 0, s, t, n_tokens, refs, add,
                            new_tokens, copy_src, copy_dst, ws);
}
qsa_status launch_pages_compact(const PageTable &t, const int32_t *refs, int32_t *table_out, int32_t *refs_out,
                                int32_t *copy_src, int32_t *copy_dst, const PagesWs &ws, cudaStream_t s) {
    const qsa_status st = launch_dependent("pages_compact_kernel launch", pages_compact_kernel, 1, kOneThreads, 0, s, refs,
                                           t.n_pages, refs_out, copy_src, copy_dst, ws);
    if (st != QSA_OK) return st;
    const long long ctas = ((long long)t.n_rows * t.max_pages + kRowThreads - 1) / kRowThreads, most = 8ll * num_sms();
    return launch_dependent("pages_retable_kernel launch", pages_retable_kernel, (int)(ctas < most ? ctas : most), kRowThreads,
                            0, s, t, table_out, ws);
}
qsa_status launch_pages_append(const PageTable &t, const PagesAppendArgs &a, cudaStream_t s) {
    // a row's entries touch at most one page per 64 and two more, and no more pages than entries
    long long units = a.n / 64 + 2ll * t.n_rows;
    if (units > a.n) units = a.n;
    cudaLaunchConfig_t cfg{};
    // A CTA looks its page up once for all heads, unless the GPU would stay empty (us, so / a head each always: 4,000 rows of one
    // token, 8 heads 132 / 401, 131,072 tokens in one row, 4 heads 82 / 79; all heads always: 8 rows of 16 tokens 3.6 / 8.0)
    const long long spread = 8ll * num_sms() / units;
    cfg.gridDim = dim3((unsigned)units, (unsigned)(spread < 1 ? 1 : spread < a.n_kv_heads ? spread : a.n_kv_heads));
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, pages_append_kernel, t, a), "pages_append_kernel launch");
}

}  // namespace qsa
