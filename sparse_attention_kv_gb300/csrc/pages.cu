// pages.cu -- the pages of a 16-bit cache shared by many sequences: fork, release, reserve, compact and append
// (the copy of whole pages is gather_blocks_kernel's).
//
// What a page's entry in a table says is in qsa.h.  The bookkeeping reads and writes a few KB, so its time is a launch
// and a chain of loads; what there is to choose is the number of steps in that chain.
//  - fork, release: one CTA per row, references by atomics (integers: any order gives the same).
//  - reserve: one CTA.  A warp counts what a row lacks; shared last pages are settled by rank among the rows that write
//    (a row copies when more references than rows before it remain); one scan gives each row its part of the ascending list of
//    free pages, and a warp fills the row's entries from it.  The list is written no further than it is needed.
//  - compact: one CTA lists the free pages below the number of live ones and the live pages behind it, both in order,
//    and pairs them; a second grid rewrites the table.
//  - append: one CTA per (page touched, KV head): K rows as they are, V through shared memory into its dimension-major block.
#include <cstdint>

#include "launch.h"
#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int kRowThreads = 256;    // fork, release, append
constexpr int kOneThreads = 1024;   // reserve, compact

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
__device__ __forceinline__ void give_back(int32_t *refs, int page, uint32_t *flags) {
    if (atomicSub(refs + page, 1) <= 0) {   // nothing refers to it: as before
        atomicAdd(refs + page, 1);
        raise(flags, QSA_FLAG_BAD_ID);
    }
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
        if (had >= 0 && had < t.n_pages) give_back(refs, had, t.flags);
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
    for (int j = (int)(((unsigned)left + 63u) >> 6) + tid; j < t.max_pages; j += kRowThreads) {
        const int page = a[j];
        if (page == -1) continue;
        if (page < 0 || page >= t.n_pages) {
            raise(t.flags, QSA_FLAG_BAD_ID);
            continue;
        }
        give_back(refs, page, t.flags);
        a[j] = -1;
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
enum : uint8_t { kWhole = 0, kCopies = 1, kKeeps = 2, kPast = 3 };

__global__ void __launch_bounds__(kOneThreads) pages_reserve_kernel(PageTable t, const int32_t *n_tokens, int32_t *refs,
                                                                    const int32_t *add, int32_t *new_tokens,
                                                                    int32_t *copy_src, int32_t *copy_dst, PagesWs ws) {
    __shared__ int32_t last[QSA_MAX_TABLE_ROWS];   // the page a row is about to write into, or -1
    __shared__ uint8_t what[QSA_MAX_TABLE_ROWS];
    __shared__ unsigned long long sums[kOneThreads / 32];
    __shared__ int counts[kOneThreads / 32];
    wait_prior_grid();
    allow_dependent_launch();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const long long most = 64ll * t.max_pages;
    // what each row lacks
    for (int row = wid; row < t.n_rows; row += kOneThreads / 32) {
        const int n = n_tokens[row];
        int more = add[row];
        if (more < 0) {
            if (lane == 0) raise(t.flags, QSA_FLAG_NBLOCKS_CLAMPED);
            more = 0;
        }
        const bool past = n < 0 || (long long)n + more > most;
        int lacks = 0, page = -1;
        if (!past && more > 0) {
            const int32_t *a = t.table + (size_t)row * t.stride;
            const int b0 = (n + 63) >> 6, b1 = (int)(((long long)n + more + 63) >> 6);
            for (int b = b0 + lane; b < b1; b += 32) {
                const int p = a[b];
                if (p >= t.n_pages || p < -1) raise(t.flags, QSA_FLAG_BAD_ID);
                lacks += p < 0 || p >= t.n_pages;
            }
            lacks = __reduce_add_sync(~0u, lacks);
            if (n & 63) {
                page = a[n >> 6];
                if (page < 0 || page >= t.n_pages) {   // a page that the tokens should have lain in
                    if (lane == 0) raise(t.flags, QSA_FLAG_BAD_ID);
                    page = -1;
                    ++lacks;
                }
            }
        }
        if (lane == 0) {
            if (past) raise(t.flags, QSA_FLAG_NBLOCKS_CLAMPED);
            last[row] = page;
            what[row] = past ? kPast : kWhole;
            ws.need[row] = lacks;
        }
    }
    __syncthreads();
    // rows that share their last page: the k-th of them to write copies while more than k references remain
    for (int row = tid; row < t.n_rows; row += kOneThreads) {
        const int page = last[row];
        if (page < 0) continue;
        const int held = refs[page];
        if (held <= 1) continue;
        int earlier = 0;
        for (int j = 0; j < row; ++j) earlier += last[j] == page;
        const bool copies = held - earlier > 1;
        what[row] = copies ? kCopies : kKeeps;
        if (copies) ws.need[row] += 1;
    }
    __syncthreads();
    // pages that a row and those before it ask for
    unsigned long long asked = 0ull;
    for (int r0 = 0; r0 < t.n_rows; r0 += kOneThreads) {
        const int row = r0 + tid;
        unsigned long long total;
        const unsigned long long incl = scan_all(row < t.n_rows ? (unsigned long long)ws.need[row] : 0ull, sums, total);
        if (row < t.n_rows) {   // more than a pool holds is more than is free
            const unsigned long long upto = asked + incl;
            ws.need[t.n_rows + row] = (int)(upto < (1ull << 30) ? upto : (1ull << 30));
        }
        asked += total;
    }
    const int want = (int)(asked < (unsigned long long)t.n_pages ? asked : (unsigned long long)t.n_pages);
    // the first free pages in order, as many as are asked for
    int free_pages = 0;
    for (int p0 = 0; p0 < t.n_pages && free_pages < want; p0 += 4 * kOneThreads) {
        int mine[4], k = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = p0 + tid * 4 + e;
            mine[e] = p < t.n_pages ? refs[p] : 1;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) k += mine[e] == 0;
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
            if (mine[e] == 0) {
                if (at < want) ws.list[at] = p0 + tid * 4 + e;
                ++at;
            }
    }
    __syncthreads();   // the list and the rows' needs lie in global memory, read by other threads of this CTA
    for (int row = wid; row < t.n_rows; row += kOneThreads / 32) {
        const int n = n_tokens[row], more = max(add[row], 0), need = ws.need[row], upto = ws.need[t.n_rows + row];
        const uint8_t does = what[row];
        const bool served = does != kPast && (upto <= free_pages || (need == 0 && does != kKeeps));
        int from = -1, to = -1;
        if (served && need > 0) {
            int32_t *a = t.table + (size_t)row * t.stride;
            int at = upto - need;
            int b = (n + 63) >> 6;
            const int b1 = (int)(((long long)n + more + 63) >> 6);
            if ((n & 63) && (does == kCopies || last[row] < 0)) {   // the page under the last tokens comes first
                to = ws.list[at];
                if (does == kCopies) from = last[row];
                if (lane == 0) {
                    a[n >> 6] = to;
                    refs[to] = 1;
                    if (from >= 0) atomicSub(refs + from, 1);
                }
                if (from < 0) to = -1;   // nothing to copy
                ++at;
            }
            for (; b < b1; b += 32) {
                const bool in = b + lane < b1;
                const int p = in ? a[b + lane] : 0;
                const bool lacks = in && (p < 0 || p >= t.n_pages);
                const unsigned who = __ballot_sync(~0u, lacks);
                if (lacks) {
                    const int page = ws.list[at + __popc(who & ((1u << lane) - 1u))];
                    a[b + lane] = page;
                    refs[page] = 1;
                }
                at += __popc(who);
            }
        }
        if (lane == 0) {
            if (!served && does != kPast) raise(t.flags, QSA_FLAG_NO_PAGES);
            new_tokens[row] = served ? n + more : n;
            copy_src[row] = from;
            copy_dst[row] = to;
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

// Exclusive and total sums of a per-row count over the CTA, for the row that holds unit `unit`.
struct Unit {
    int row, index;   // the index-th page that the row's entries touch; row < 0: no such unit
};
struct Span {
    int e0;            // first entry
    long long lo, hi;  // positions
    int first;
};
__device__ __forceinline__ Span span_of(const PageTable &t, const PagesAppendArgs &a, int row, bool tell) {
    Span s;
    int c0 = a.cu_rows[row], c1 = a.cu_rows[row + 1];
    if (tell && (c0 < 0 || c0 > a.n || c1 < c0 || c1 > a.n)) raise(t.flags, QSA_FLAG_NBLOCKS_CLAMPED);
    c0 = min(max(c0, 0), a.n);
    c1 = min(max(c1, c0), a.n);
    s.e0 = c0;
    s.first = a.first[row];
    const long long end = (long long)s.first + (c1 - c0), most = 64ll * t.max_pages;
    s.lo = s.first < 0 ? 0 : s.first;
    s.hi = end > most ? most : end;
    if (tell && c1 > c0 && (s.first < 0 || end > most)) raise(t.flags, QSA_FLAG_NBLOCKS_CLAMPED);
    if (s.hi < s.lo || c1 == c0) s.hi = s.lo;
    return s;
}
__device__ __forceinline__ int pages_of(const Span &s) { return s.hi > s.lo ? (int)(((s.hi + 63) >> 6) - (s.lo >> 6)) : 0; }

__global__ void __launch_bounds__(kRowThreads) pages_append_kernel(PageTable t, PagesAppendArgs a) {
    __shared__ BlockScratch sm;
    __shared__ Unit unit;
    __shared__ __align__(16) uint16_t tile[64][136];   // V rows; 272 bytes a row: 16-byte aligned
    __shared__ int source[64];
    wait_prior_grid();
    allow_dependent_launch();
    const int tid = threadIdx.x, g = blockIdx.y;
    if (tid == 0) unit.row = -1;
    __syncthreads();
    int before = 0;
    for (int r0 = 0; r0 < t.n_rows && before <= (int)blockIdx.x; r0 += kRowThreads) {
        const int row = r0 + tid;
        const int np = row < t.n_rows ? pages_of(span_of(t, a, row, blockIdx.x == 0 && g == 0)) : 0;
        int total;
        const int at = before + block_excl_scan<kRowThreads>(np, sm, total);
        if ((int)blockIdx.x >= at && (int)blockIdx.x < at + np) {
            unit.row = row;
            unit.index = (int)blockIdx.x - at;
        }
        before += total;
    }
    __syncthreads();
    const int row = unit.row;
    if (row < 0) return;
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
                if (r != -1 && g == 0) raise(t.flags, QSA_FLAG_BAD_ID);
                r = -1;
            }
        }
        source[tid] = r;
    }
    __syncthreads();
    const uint16_t *k = static_cast<const uint16_t *>(a.k.p) + (size_t)g * a.k.head;
    const uint16_t *v = static_cast<const uint16_t *>(a.v.p) + (size_t)g * a.v.head;
    uint16_t *kc = static_cast<uint16_t *>(a.kcache) + ((size_t)g * t.n_pages + page) * (64 * 128);
    uint16_t *vc = static_cast<uint16_t *>(a.vcache_t) + ((size_t)g * t.n_pages + page) * (64 * 128);
    const int c = tid & 15;
    uint4 kx[4], vx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = source[(tid >> 4) + 16 * i];
        kx[i] = vx[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= 0) {
            kx[i] = *reinterpret_cast<const uint4 *>(k + (int64_t)r * a.k.token + 8 * c);
            vx[i] = *reinterpret_cast<const uint4 *>(v + (int64_t)r * a.v.token + 8 * c);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = (tid >> 4) + 16 * i;
        if (source[at] >= 0) *reinterpret_cast<uint4 *>(kc + at * 128 + 8 * c) = kx[i];
        *reinterpret_cast<uint4 *>(&tile[at][8 * c]) = vx[i];
    }
    __syncthreads();
    // dimension d, eight tokens a thread; 8 lanes write a dimension's 128 bytes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = (tid >> 3) + 32 * i, t0 = (tid & 7) * 8;
        uint16_t x[8];
        bool all = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = tile[t0 + j][d];
            all = all && source[t0 + j] >= 0;
        }
        if (all) {
            *reinterpret_cast<uint4 *>(vc + d * 64 + t0) =
                make_uint4(x[0] | (uint32_t)x[1] << 16, x[2] | (uint32_t)x[3] << 16, x[4] | (uint32_t)x[5] << 16,
                           x[6] | (uint32_t)x[7] << 16);
        } else {
            for (int j = 0; j < 8; ++j)
                if (source[t0 + j] >= 0) vc[d * 64 + t0 + j] = x[j];
        }
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
    cfg.gridDim = dim3((unsigned)units, (unsigned)a.n_kv_heads);
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
