// dense_attn.cu -- attention of whole prompts over packed rows, and of drafted token trees over pages.
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale (s_t - m)),  s_t = q . k_t,
//
// over the keys t that a row (a query token under one head) sees: causal ones of packed rows, or the pages of a
// sequence and the row's ancestors among the drafts.  One pass over the keys, 128 a step, with a running reference m:
//   S = Q K^T   tcgen05, M = 128 rows, N = 128 keys, into tensor memory
//   P = exp2    one thread per row reads its 128 logits, writes the weights in 16 bits over them in tensor memory
//   O += P V    tcgen05 with A = P from tensor memory, M = 128 rows, N = 128 dimensions
// The rows of a stream are (token, head of the group) pairs, token-major, 128 / group whole tokens: all rows share one KV
// head's K and V, a tile of two streams spans few tokens (16 at groups of 16), so that little of a causal tile is masked, and
// a single token's 16 heads read a page once.  A CTA works on both streams in turn: the tensor cores multiply for
// one while the other's softmax runs, and both take the same K and V from shared memory.  Where no sequence fills more than
// one stream (a decode step) both take the same rows and half of a step's keys each, and are joined at the end.
// m moves only when a row's maximum has risen by more than 2^8 of weight (then l and O are scaled in place): any
// reference gives the same quotient, sums stay below 2^8 x keys, weights keep their relative precision.
// The product with V takes the weights in V's 16 bits, as kind::f16 wants its A; l sums them before that rounding, since lse comes
// from l too and would be off by up to half a step of that type.  So a row that one key outweighs, whose weight is no power
// of two (it came after m was set), has V off by that much (2^-8 bf16, 2^-11 fp16), in an fp32 out as well; over many keys it averages out.
//
// Work: every (sequence, KV head, tile) is a run of steps; a persistent grid of one CTA per SM takes the runs whole or in
// pieces (see Walk).  A run in pieces is joined by combine_kernel from the CTAs' partial (O, m, l).
//
// Roles: warp 0 finds the pieces, publishes them and copies (TMA; a ring of 32 KB slots, K and V in turn), warps 1 and 2
// issue a stream's products, warp 3 clears values, warps 4-7 and 8-11 are a stream's softmax and epilogue.  V of packed
// rows is an MN-major operand, V of a page a K-major one (its dimension comes before its token).
// Values at places that a row does not see must not reach it as 0 x NaN: in steps that hold such places warp 3 clears what
// lies past the last row's view and any value that is not finite; the latter is added at the end to the rows that see it.
//
// What bounds it.  Prompts: the tensor cores, and the power limit when calls last.  A step of 256 rows and 128 keys is 2,048
// cycles of MMA; it takes 2,150 to 2,350 (1.1-1.2 us at 1.95 GHz), the rest being the chain P ready -> P V -> S -> softmax
// (0.5 us) of a stream where it does not fit beside the other one's products.  256 queries x 64 heads behind 130,816 tokens: 0.56 ms
// in a burst (1.96 PFLOP/s), 0.64 sustained; one prompt of 16,384 tokens, 64 heads in 4 groups: 2.18 (2.01) and 2.5 ms (a large
// library product 1.88 and 1.72 PFLOP/s here).  Decode: HBM; one query at 258,000 tokens, 64 heads in 4 groups: 94-98 us, of which
// 88 the main kernel (528 MB, 6.0 TB/s).  Short calls: about 13 us for a CTA's first piece (2 to find it, 2 until its first
// product, 2.2 for its end), 4.4 us for a further one of a single step.
// Measured on the way (16,384 tokens, ms): one warp issuing both streams, descriptors made in divergent code 5.19 (an MMA then
// takes about 100 cycles to issue); Q by TMA, outputs in whole rows 3.81; two threads a row, two issuing warps in turn,
// descriptors in uniform registers 2.86; a thread a row, weights passed on in two parts 2.70; steps that are not seen whole in
// rolled loops (instruction fetches) 2.55; runs dealt out 2.48; fewer registers held over a step 2.30.
//
// Every wait is bounded; on expiry the CTA raises QSA_FLAG_WAIT_TIMEOUT, drains its copies and MMAs, frees its tensor memory
// and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "launch.h"
#include "qsa_device.cuh"
#include "qsa_internal.h"
#include "tc_ptx_tmem.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;         // a thread a row
constexpr int kRows = 128;            // rows of a stream (TMEM lanes)
constexpr int kKeys = 128;            // keys of a step
constexpr int kSlots = 4;
constexpr int kSlotBytes = kKeys * 128 * 2;
constexpr int kQBytes = kRows * 128 * 2;
constexpr int kStageBytes = 4096;     // per softmax warp: 32 rows of 128 bytes on their way out
constexpr int kPieces = 4;            // pieces that are published ahead
constexpr int kInfo = 8;              // steps whose page limits are held: more than the ring holds
constexpr int kMaxCtas = 152;
// How runs are shared out (measured in us, this side / the other):
constexpr int kWhole = 8;       // runs of up to 8 steps are not split (4: a split one of 5 steps 15 / 18; 16: one of 12 steps 17 / 22)
constexpr int kLeast = 3;       // steps of a piece of the others, at least (17 steps: in 3s 17.5, in 6s 19.6, in 2s 17.7)
constexpr int kSlack = 4;       // steps that pieces of one length may lie above an even share (6 above: 64 nodes at 131,072 tokens 174 / 180)
constexpr int kRunKeys = 512;   // what a run's beginning and end cost, in keys (1024: 4,096 tokens 206 / 193, a mixed batch 270 / 304; 256: 206 / 239)
constexpr int kTable = 256;     // sequences whose runs are counted in shared memory
constexpr int kShortRun = 16;   // steps of runs that are dealt out however few the shares hold (0: 1,024 tokens 29 / 35; 64: no better)
constexpr int kMinShare = 384;  // work, in keys, for each share that is used, the last one's rounded up: they hold half of it each at least
constexpr int kShortKeys = 2048; // a sequence's keys up to which rows leave by TMA: see launch()
constexpr int kManyParts = 8;   // parts of a run that combine_kernel shares out to its warps (38 parts 94 / 102; 64 sequences' two or three 360 / 348)
// The join takes a share without a part for its run's end: borders a step apart have another step begin nearest to them.
static_assert(kMinShare / 2 >= kKeys, "a share in the middle of a run has a step of it");
constexpr float kRise = 8.0f;         // log2 of the largest weight before the reference moves
constexpr uint32_t kColO = 0, kColS = 256;   // + 128 x stream

struct Params {
    Rows16 v;
    const int32_t *cu_q, *cu_k;
    int n_seqs, total_q, total_k;
    int n_heads, n_kv, group;
    int toks;             // tokens of a stream: 128 / group, so that a stream begins with a token
    int tile;             // tokens of a tile: two streams', or one's where both take the same
    uint32_t by_group;    // ceil(2^16 / group): x / group = x * by_group >> 16 for x < 128
    float scale, scale_log2;
    void *out;
    int out_f32;
    float *lse;
    const int32_t *parents;
    int max_nodes;
    const int32_t *table;
    int64_t table_stride;
    int max_pages, n_pages;
    const int32_t *n_tokens;
    int row_tiles;        // trees: CTAs side by side that take a tile of rows each
    int shares;           // CTAs (or groups of row_tiles) that take a share
    int rows_cap;         // rows of a partial
    float4 *part;         // [grid][2][32][rows_cap]: O, four dimensions of a row at a time
    float2 *ml;           // [grid][2][rows_cap]: (m scale log2 e, l)
    int4 *desc;           // [grid][2]: see describe()
    unsigned *dealt;      // runs dealt out so far, and CTAs that are done; both 0 between calls
    uint32_t *flags;
};

// What a CTA works on at a time: steps s0 .. s1 - 1 of a run's n, for a tile.
struct Piece {
    int stop;             // no piece: the CTA is done
    int bad;              // a value in a step that not every row sees whole was not finite
    int s, g;
    int q0, lq, k0, lk;
    int tok0;             // the tile's first token in its sequence
    int s0, s1, n;
    int first;            // the step it begins with: first .. s1 - 1, then s0 .. first - 1
    int rows[2];          // rows of each stream
    int e[2];             // where each stream's steps end (<= s1; s0: none)
};

// The step in a piece's order that stands at place j of s0 .. s1 - 1.
__device__ __forceinline__ int step_at(int j, int s0, int s1, int first) {
    const int x = j + first - s0;
    return x < s1 ? x : x - (s1 - s0);
}

struct Ctrl {
    uint64_t full[kSlots], empty[kSlots], clean[kSlots / 2], turn[2];
    uint64_t qfull[2], qempty[2], sfull[2], pready[2][2], ofull[2];
    uint64_t pfull[kPieces], pempty[kPieces];
    uint64_t drain[2];
    Piece pieces[kPieces];
    uint32_t tmem;
    int abort;
    int2 info[kInfo];     // valid tokens in each page of a step
    float2 other[kRows];  // HALVES: stream 1's (m, l)
    int runs[kTable + 1]; // runs of the sequences before each one
    int dealing;          // the CTAs take runs as they come free
};
constexpr int kOffQ = 0;
constexpr int kOffRing = 2 * kQBytes;
constexpr int kOffStage = kOffRing + kSlots * kSlotBytes;
constexpr int kOffCtrl = kOffStage + kSoftWarps * kStageBytes;
constexpr int kSmem = kOffCtrl + (int)sizeof(Ctrl);
static_assert(kSmem <= 232448, "shared memory");

__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
    const unsigned long long t0 = now_ns();
    while (true) {
        if (__all_sync(~0u, mbar_try_wait_sleep(bar, parity))) return true;
        if (__any_sync(~0u, *abort_flag != 0)) return false;
        if (__any_sync(~0u, now_ns() - t0 > kWaitNs)) {
            *abort_flag = 1;
            return false;
        }
    }
}

// The same value in every lane, so that the compiler may hold it (and what follows from it) once per warp: the descriptors of
// the products are taken from uniform registers, and moving them there for each one takes longer than forming it.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(~0u, x, 0); }
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}
// Whether x holds in any of `threads` threads, which meet at barrier `id`.
__device__ __forceinline__ bool any_of(int id, int threads, bool x) {
    int any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((int)x), "r"(id), "r"(threads)
        : "memory");
    return any != 0;
}
// HALVES: the two warps that hold a row's halves, one of each stream.
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync %0, 64;" ::"r"(4 + (threadIdx.x >> 5 & 3)) : "memory"); }

// ------------------------------------------------------------------ the runs and the shares

// a b / c: by 32-bit division where the sizes allow
__device__ __forceinline__ long long mul_div(unsigned a, long long b, unsigned c) {
    return b < (1 << 24) ? (long long)(a * (unsigned)b / c) : (long long)a * b / c;   // a, c <= 152
}

template <bool TREE>
struct Seq {
    int q0, lq, k0, lk, tiles;   // trees: lk = tokens in the pages

    __device__ __forceinline__ void load(const Params &p, int s, bool tell) {
        range(p, p.cu_q, s, p.total_q, tell, q0, lq);
        if constexpr (TREE) {
            if (lq > p.max_nodes) {
                lq = p.max_nodes;
                if (tell) atomicOr(p.flags, QSA_FLAG_NBLOCKS_CLAMPED);
            }
            const int n = p.n_tokens[s], most = 64 * p.max_pages;
            lk = min(max(n, 0), most);
            if (tell && lk != n) atomicOr(p.flags, QSA_FLAG_NBLOCKS_CLAMPED);
            k0 = 0;
            tiles = lq > 0 ? 1 : 0;   // each CTA of a group has its own tile of rows
        } else {
            range(p, p.cu_k, s, p.total_k, tell, k0, lk);
            tiles = (lq + p.tile - 1) / p.tile;
        }
    }
    static __device__ __forceinline__ void range(const Params &p, const int32_t *cu, int s, int most, bool tell, int &c0,
                                                 int &len) {
        const int a = cu[s], b = cu[s + 1];
        if (tell && (a < 0 || b < a || b > most)) atomicOr(p.flags, QSA_FLAG_NBLOCKS_CLAMPED);
        c0 = min(max(a, 0), most);
        len = min(max(b, c0), most) - c0;
    }
    // What lane l of the warp has loaded.
    __device__ __forceinline__ void take(const Seq &x, int l) {
        q0 = __shfl_sync(~0u, x.q0, l);
        lq = __shfl_sync(~0u, x.lq, l);
        k0 = __shfl_sync(~0u, x.k0, l);
        lk = __shfl_sync(~0u, x.lk, l);
        tiles = __shfl_sync(~0u, x.tiles, l);
    }
    __device__ __forceinline__ int steps(const Params &p, int t) const {
        if constexpr (TREE) return (lk + kKeys - 1) / kKeys + 1;   // the pages, then the drafts
        return (keys_of(lq, lk, min((t + 1) * p.tile, lq) - 1) + kKeys - 1) / kKeys;
    }
    // The work of tiles 0 .. T - 1, in keys: what each tile's last token sees, and kRunKeys.  With W tokens a tile, that is
    // max(0, lk - lq + (t + 1) W) for a full tile t; the last one's is lk.
    __device__ __forceinline__ long long cum(const Params &p, int T) const {
        if constexpr (TREE) return T ? lk + kKeys + kRunKeys : 0;
        long long sum = (long long)T * kRunKeys;
        if (T == tiles && T > 0) {
            sum += lk;
            --T;
        }
        const int W = p.tile, c = lk - lq + W, t0 = c < 0 ? min((-c + W - 1) / W, T) : 0;
        const long long n = T - t0;
        return sum + n * (c + (long long)t0 * W) + W * (n * (n - 1) / 2);
    }
    __device__ __forceinline__ int work(const Params &p, int t) const {   // cum(t + 1) - cum(t)
        if constexpr (TREE) return lk + kKeys + kRunKeys;
        return keys_of(lq, lk, min((t + 1) * p.tile, lq) - 1) + kRunKeys;
    }
    // Keys that token i of lq sees.
    static __device__ __forceinline__ int keys_of(int lq, int lk, int i) { return min(max(lk - lq + i + 1, 0), lk); }
};

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}
__device__ __forceinline__ int warp_scan(int v) {   // inclusive
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(~0u, v, d);
        if ((int)(threadIdx.x & 31) >= d) v += x;
    }
    return v;
}

// A CTA's pieces one after another (one warp).  Which they are goes by one of three rules, the same in every CTA:
//  kEven   no more runs than shares: each run in equal pieces, a share each, where that costs little against an even split
//  kDealt  more runs, those that end last short against a share: whole, longest first within a (sequence, KV head), each to the
//          next CTA that is free
//  kBorder otherwise: all runs laid end to end and cut at equal distances
// Measured, us: kEven / kBorder, 5 trees over 900 tokens 24 / 30; kDealt / kBorder, a prompt of 1,024 tokens 27 / 34, of 2,600
// 85 / 97, of 16,384 2,213 / 2,280, 40 decodes of 2,500 tokens (8 heads; taken by kBorder) 104 / 88.
enum Rule { kEven, kDealt, kBorder };

template <bool TREE, bool HALVES>
struct Walk {
    Seq<TREE> q;
    Rule rule;
    int s, g, t, tile;
    long long at, x0, x1;   // kBorder: the beginning of the next run (from the last one down), and the CTA's share of all runs
    int period, done;       // and steps of a share, steps taken
    int run, runs;          // kDealt: the next run, more runs than shares
    bool begun;
    Seq<TREE> mine;         // up to 32 sequences: a lane each
    int s0, s1;             // kEven: the piece's steps; s0 < 0: no piece (any more)

    // The piece s0 .. s1 - 1 of the run (s, g, t); false when this CTA has no rows in it.
    __device__ __forceinline__ bool fill(const Params &p, Piece &pc, int from, int to, int n) const {
        pc.s = s;
        pc.g = g;
        pc.q0 = q.q0;
        pc.lq = q.lq;
        pc.k0 = q.k0;
        pc.lk = q.lk;
        pc.tok0 = (TREE ? tile : t) * p.tile;
        pc.s0 = from;
        pc.s1 = to;
        pc.n = n;
        pc.first = from;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int first = pc.tok0 + (HALVES ? 0 : i * p.toks), toks = min(max(q.lq - first, 0), p.toks);
            pc.rows[i] = toks * p.group;
            int end = from;
            if (toks > 0) {
                end = TREE ? n : (q.keys_of(q.lq, q.lk, first + toks - 1) + kKeys - 1) / kKeys;
                end = max(min(end, to), from);
            }
            pc.e[i] = end;
        }
        return pc.tok0 < q.lq;
    }
    // Run i of all: by sequence, KV head, tiles from the last one on.  Every lane calls, for a run of its own.
    __device__ __forceinline__ void locate(const Params &p, const Ctrl &ct, int i) {
        int lo = 0, hi = p.n_seqs;   // runs[lo] <= i < runs[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (ct.runs[mid] <= i) lo = mid;
            else hi = mid;
        }
        s = lo;
        __syncwarp();
        if (p.n_seqs <= 32) q.take(mine, lo);
        else q.load(p, lo, false);
        const int local = i - ct.runs[lo], tiles = max(q.tiles, 1);
        g = local / tiles;
        t = tiles - 1 - (local - g * tiles);
    }
    __device__ __forceinline__ bool next(const Params &p, const Ctrl &ct, Piece &pc) {
        if (rule == kEven) {
            if (s0 < 0) return false;
            const int from = s0;
            s0 = -1;
            return fill(p, pc, from, s1, q.steps(p, t));
        }
        if (rule == kDealt) {
            while (run < runs) {
                if (begun) {   // the copies of the run before are on their way
                    unsigned i = 0;
                    if ((threadIdx.x & 31) == 0) i = atomicAdd(p.dealt + 2 * tile, 1u);
                    i = __shfl_sync(~0u, i, 0);
                    if (i >= (unsigned)(runs - p.shares)) break;
                    run = p.shares + (int)i;
                }
                begun = true;
                locate(p, ct, run);
                const int n = q.steps(p, t);
                if (fill(p, pc, 0, n, n)) return true;
            }
            return false;
        }
        while (s >= 0) {
            const int n = q.steps(p, t), work = q.work(p, t);
            const long long from = at;
            if (from + work <= x0) break;
            int a0 = 0, a1 = n;
            bool take = from >= x0;
            if (n > kWhole) {   // the step that begins nearest to a border; both sides of it compute the same
                const long long a = (x0 - from - kRunKeys + kKeys / 2) / kKeys, b = (x1 - from - kRunKeys + kKeys / 2) / kKeys;
                a0 = x0 <= from || a <= 0 ? 0 : (int)(a < n ? a : n);
                a1 = b <= 0 ? 0 : b < n && x1 < from + work ? (int)b : n;
                take = a1 > a0;
            }
            take = fill(p, pc, a0, a1, n) && take;
            if (!TREE && take) {
                // Runs of one KV head lie at all distances from one another, so that CTAs which began at their shares' beginnings
                // would read all keys over and over from HBM.  Each takes the step that the others take now, modulo the
                // share, if it has it (where both streams see all of the piece).
                int r = (done - a0) % period;
                if (r < 0) r += period;
                if (a0 + r < a1 && (pc.e[0] == a1 || pc.e[0] == a0) && (pc.e[1] == a1 || pc.e[1] == a0)) pc.first = a0 + r;
                done += a1 - a0 + kRunKeys / kKeys;
            }
            if (--t < 0) {
                if (--g < 0) {
                    do {
                        if (--s < 0) break;
                        q.load(p, s, false);
                    } while (q.tiles == 0);
                    g = p.n_kv - 1;
                }
                t = q.tiles - 1;
            }
            if (s >= 0) at -= q.work(p, t);
            if (take) return true;
        }
        return false;
    }
};

// The rule, and where this CTA begins (one warp).
template <bool TREE, bool HALVES>
__device__ void find_share(const Params &p, Ctrl &ct, Walk<TREE, HALVES> &w) {
    const int lane = threadIdx.x & 31;
    const unsigned share = blockIdx.x / (unsigned)p.row_tiles;
    const bool tell = blockIdx.x == 0, counted = p.n_seqs <= kTable;
    Seq<TREE> &q = w.q;
    auto weight = [&](int s, bool say) -> long long {
        if (s >= p.n_seqs) {
            q = Seq<TREE>{};
            return 0;
        }
        q.load(p, s, say);
        return p.n_kv * q.cum(p, q.tiles);
    };
    long long total = 0, first = 0, rows = 0;   // first: the weights of sequences 0 .. 31
    int runs = 0, longest = 0;
    Seq<TREE> last{};   // that has queries
    for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
        const long long x = weight(s0 + lane, tell);
        if (s0 == 0) {
            first = x;
            w.mine = q;
        }
        total += warp_sum(x);
        rows += warp_sum(q.lq);
        const bool in = s0 + lane < p.n_seqs;
        longest = max(longest, in && q.tiles > 0 ? q.work(p, q.tiles - 1) : 0);
        if (counted) {
            const int mine = in ? p.n_kv * q.tiles : 0, incl = warp_scan(mine);
            if (in) ct.runs[s0 + lane + 1] = runs + incl;
            runs += __shfl_sync(~0u, incl, 31);
            const unsigned some = __ballot_sync(~0u, q.tiles > 0);
            if (some) last.take(q, 31 - __clz(some));
        }
    }
    longest = __reduce_max_sync(~0u, longest);
    if (lane == 0) ct.runs[0] = 0;
    __syncwarp();
    w.tile = TREE ? (int)(blockIdx.x % (unsigned)p.row_tiles) : 0;
    w.rule = kBorder;
    if (rows > p.total_q) {   // sequences that overlap would write rows twice, and be any amount of work: nothing is done
        if (tell && lane == 0) atomicOr(p.flags, QSA_FLAG_NBLOCKS_CLAMPED);
        w.rule = kEven;
        w.s0 = -1;
        return;
    }
    if (counted && runs <= p.shares) {
        constexpr int kTurns = (kMaxCtas + 31) / 32;
        int n[kTurns], steps = 0;
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int i = lane + 32 * k;
            n[k] = 0;
            if (32 * k < runs) {
                w.locate(p, ct, min(i, runs - 1));
                if (i < runs) n[k] = max(q.steps(p, w.t), 1);
            }
            steps += n[k];
        }
        steps = __reduce_add_sync(~0u, min(steps, 1 << 24));
        const int even = (steps + p.shares - 1) / p.shares;
        int len = max(even, kLeast);   // of a piece, at most
        auto pieces_of = [&](int n) { return n <= kWhole ? min(n, 1) : (n + len - 1) / len; };
        const int most = len + kSlack;
        while (len <= most) {
            int pieces = 0;
#pragma unroll
            for (int k = 0; k < kTurns; ++k) pieces += pieces_of(n[k]);
            if (__reduce_add_sync(~0u, pieces) <= p.shares) break;
            ++len;
        }
        if (len <= most) {
            w.rule = kEven;
            w.s0 = -1;
            int before = 0;
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
                const int c = pieces_of(n[k]), incl = warp_scan(c);
                const int part = (int)share - (before + incl - c);
                const unsigned mine = __ballot_sync(~0u, part >= 0 && part < c);
                if (mine) {
                    const int l = __ffs(mine) - 1, parts = __shfl_sync(~0u, c, l), of = __shfl_sync(~0u, part, l);
                    w.locate(p, ct, l + 32 * k);
                    const int all = q.steps(p, w.t);
                    w.s0 = (int)((long long)of * all / parts);
                    w.s1 = (int)((long long)(of + 1) * all / parts);
                    break;
                }
                before += __shfl_sync(~0u, incl, 31);
            }
            return;
        }
    }
    // The CTAs end within a run of the last ones dealt, one a share: of a long last sequence its first tiles, short ones
    const int tail = last.tiles > p.shares ? last.work(p, p.shares - 1) : longest;
    if (counted && runs > p.shares && tail <= max(total / p.shares / (TREE ? 3 : 2), (long long)kShortRun * kKeys + kRunKeys)) {
        w.rule = kDealt;
        w.run = (int)share;
        w.runs = runs;
        w.begun = false;
        return;
    }
    long long used = (total + kMinShare - 1) / kMinShare;
    used = used < 1 ? 1 : used > p.shares ? p.shares : used;
    w.x0 = share < used ? mul_div(share, total, (unsigned)used) : total;
    w.x1 = share < used ? mul_div(share + 1, total, (unsigned)used) : total;
    w.period = max((int)(total / used / kKeys), 1);
    w.done = 0;
    const long long x = w.x1 - 1;   // in the share's last run
    long long before = 0;
    w.at = w.x0;
    w.s = -1;
    w.g = w.t = 0;
    for (int s0 = 0; s0 < p.n_seqs && w.x0 < w.x1; s0 += 32) {
        const long long y = s0 == 0 && p.n_seqs <= 32 && runs > p.shares ? first : weight(s0 + lane, false);
        long long incl = y;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long z = __shfl_up_sync(~0u, incl, d);
            if (lane >= d) incl += z;
        }
        const unsigned past = __ballot_sync(~0u, before + incl > x);
        if (past) {
            const int l = __ffs(past) - 1;
            w.s = s0 + l;
            before += __shfl_sync(~0u, incl - y, l);
            break;
        }
        before += __shfl_sync(~0u, incl, 31);
    }
    if (w.s >= 0) {
        q.take(q, w.s & 31);
        const long long per = q.cum(p, q.tiles), in_seq = x - before;
        w.g = in_seq < (1ll << 31) && per < (1ll << 31) ? (int)((unsigned)in_seq / (unsigned)per) : (int)(in_seq / per);
        before += w.g * per;
        int lo = 0, hi = q.tiles;   // cum(lo) <= x - before < cum(hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, mid = min(lo + (lane + 1) * step, hi);
            const unsigned over = __ballot_sync(~0u, q.cum(p, mid) > x - before);   // lane 31 reaches hi
            const int l = __ffs(over) - 1;
            const int new_hi = min(lo + (l + 1) * step, hi);
            lo += l * step;
            hi = new_hi;
        }
        w.t = lo;
        w.at = before + q.cum(p, lo);
    }
}

// ------------------------------------------------------------------ arithmetic

using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t r;
    if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool F16>
__device__ __forceinline__ float widen(uint32_t half) {
    if constexpr (F16) return __half2float(__ushort_as_half((unsigned short)half));
    else return __uint_as_float(half << 16);
}
// Bits of a pair of 16-bit values whose exponents are all ones: 0xFFFF where a value is not finite.
template <bool F16>
__device__ __forceinline__ uint32_t not_finite(uint32_t pair) {
    constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
    return ((pair & e) == e ? 0xFFFFu : 0u) | ((pair & (e << 16)) == (e << 16) ? 0xFFFF0000u : 0u);
}
// acc + 0 x: NaN in a half once a value there is not finite
template <bool F16>
__device__ __forceinline__ uint32_t probe(uint32_t x, uint32_t acc) {
    if constexpr (F16) asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    else asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    return acc;
}

// The nodes a tree's row sees (one warp; every lane gets its own row's): bit j of the mask is node j.
__device__ unsigned long long ancestors(const Params &p, int q0, int lq, int node) {
    const int lane = threadIdx.x & 31;
    unsigned long long mask[2];
    int up[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        int a = i < lq ? p.parents[q0 + i] : -1;
        if (a < -1 || a >= i) {
            atomicOr(p.flags, QSA_FLAG_BAD_ID);
            a = -1;
        }
        up[h] = a;
        mask[h] = 1ull << i;
    }
    auto of = [&](const unsigned long long (&m)[2], int i) {
        const unsigned long long a = __shfl_sync(~0u, m[0], i & 31), b = __shfl_sync(~0u, m[1], i & 31);
        return i & 32 ? b : a;
    };
#pragma unroll 1
    for (int round = 0; round < 6; ++round) {   // each node's mask covers 2^round nodes of its path
        unsigned long long add[2];
        int far[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = max(up[h], 0);
            add[h] = of(mask, i);
            const int a = __shfl_sync(~0u, up[0], i & 31), b = __shfl_sync(~0u, up[1], i & 31);
            far[h] = i & 32 ? b : a;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (up[h] >= 0) {
                mask[h] |= add[h];
                up[h] = far[h];
            }
    }
    return of(mask, node);
}

// ------------------------------------------------------------------ the kernel

// What a CTA left in its partials.  desc[0]: (1 = the piece ends its run, 2 = it does not, 0 = none) for a piece that began
// in an earlier CTA; desc[1]: (1, KV head, the tile's first token among all, the tokens from there to the sequence's end)
// for a run that begins here and does not end here.
__device__ __forceinline__ void describe(const Params &p, const Piece &pc) {
    int4 *d = p.desc + 2 * (size_t)blockIdx.x;
    if (pc.s0 > 0) d[0] = make_int4(pc.s1 == pc.n ? 1 : 2, 0, 0, 0);
    else if (pc.s1 < pc.n) d[1] = make_int4(1, pc.g, pc.q0 + pc.tok0, pc.lq - pc.tok0);
}

// Four values of a row of out, at element `at`.
template <bool F16>
__device__ __forceinline__ void store4(const Params &p, size_t at, float a, float b, float c, float d) {
    if (p.out_f32) *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = make_float4(a, b, c, d);
    else *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) = make_uint2(pack16<F16>(a, b), pack16<F16>(c, d));
}

// A warp's 32 rows of out, normalised, by TMA: 32 dimensions a tile, from two buffers of the stage in turn.
template <bool F16>
__device__ __forceinline__ void tiles_out(uint32_t tO, uint8_t *stage, float inv, const CUtensorMap *tm_o, int head, int token) {
    int lane;
    asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));   // so that nothing that follows from it is held over the steps
#pragma unroll 1
    for (int d = 0; d < 128; d += 32) {
        uint32_t o[2][16];
        tmem_ld16_nowait(tO + d, o[0]);
        tmem_ld16_nowait(tO + d + 16, o[1]);
        bulk_wait_read<1>();   // the buffer that this round fills
        __syncwarp();
        tmem_wait_ld();
        reg_fence(o[0]);
        reg_fence(o[1]);
        uint8_t *buffer = stage + (d & 32) * 64;
        auto pair = [&](int i) {
            return pack16<F16>(__uint_as_float(o[i >> 4][i & 15]) * inv, __uint_as_float(o[i >> 4][(i & 15) + 1]) * inv);
        };
#pragma unroll
        for (int i = 0; i < 32; i += 8)   // the 64-byte swizzle
            *reinterpret_cast<uint4 *>(buffer + lane * 64 + (((i >> 3) ^ (lane >> 1 & 3)) << 4)) =
                make_uint4(pair(i), pair(i + 2), pair(i + 4), pair(i + 6));
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(tm_o, buffer, d, head, token);
            bulk_commit();
        }
    }
}

// The end of a piece for a warp's 32 rows: the output normalised, through `stage` so that a row's bytes are written
// together, or the partial as it is.  have: there is an O in tensor memory.
// HALVES: stream 1 hands what it has to stream 0 through `box` (32 KB), and stream 0 goes on.
// TILES: rows that are all there leave by TMA.
template <bool F16, bool TREE, bool HALVES, bool TILES>
__device__ __forceinline__ void finish(const Params &p, Ctrl &ct, const Piece &pc, bool have, uint32_t tO, uint8_t *stage, float4 *box,
                                       float m, float l, int lim, unsigned long long nodes, int rows, const CUtensorMap *tm_o) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, st = (warp - 4) >> 2, G = p.group;
    const int r = (warp & 3) * 32 + lane;
    const bool whole = pc.s0 == 0 && pc.s1 == pc.n, mine = r < rows, fix = pc.bad != 0;
    const size_t slot = 2 * (size_t)blockIdx.x + (pc.s0 > 0 ? 0 : 1);
    const int in_tile = st * kRows + r;
    // values that are not finite are added where this row sees them: in the drafts, or from the first step that was cleared
    const int f0 = TREE ? 0 : max(Seq<TREE>::keys_of(pc.lq, pc.lk, pc.tok0) / kKeys, pc.s0) * kKeys;
    const int f1 = TREE ? (pc.s1 == pc.n ? pc.lq : 0) : min(lim, pc.s1 * kKeys);
    const size_t out0 = (size_t)(pc.q0 + pc.tok0 + (HALVES ? 0 : st * p.toks)) * p.n_heads + pc.g * G;
    auto output = [&](int row) {   // the row of out that a row of the stream is
        const int tok = (int)(row * p.by_group >> 16);
        return out0 + (size_t)tok * p.n_heads + (row - tok * G);
    };
    float keep = 1.0f, add = 0.0f;   // HALVES: factors of this stream's and of the other's
    if constexpr (HALVES) {
        if (have && rows > (warp & 3) * 32) {   // the same for both warps
            if (st == 1) ct.other[r] = make_float2(m, l);
            rows_sync();
            if (st == 0) {
                const float2 x = ct.other[r];
                const float top = l == 0.0f ? x.x : x.y == 0.0f ? m : fmaxf(m, x.x);   // of those that saw something
                keep = l == 0.0f ? 0.0f : ex2((m - top) * p.scale_log2);
                add = x.y == 0.0f ? 0.0f : ex2((x.x - top) * p.scale_log2);
                m = top;
                l = keep * l + add * x.y;
            }
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if constexpr (TILES) {
        if (whole && !fix && have && rows >= (warp & 3) * 32 + 32) {
            tiles_out<F16>(tO, stage, inv, tm_o, pc.g * G, pc.q0 + pc.tok0 + st * p.toks + (int)((warp & 3) * 32 * p.by_group >> 16));
            if (p.lse) p.lse[output(r)] = l == 0.0f ? -INFINITY : m * p.scale + logf(l);
            return;
        }
        bulk_wait_read<0>();
        __syncwarp();
    }
    uint8_t *line = stage + lane * 128;
    const int unit = p.out_f32 ? 4 : 2;
    // 32 dimensions a round: in 16 bits two rounds make 128 bytes of each row, in 32 bits one
#pragma unroll 1
    for (int d = 0; d < 128; d += 32) {
        uint32_t o[2][16];
        __syncwarp();
        if (have) {
            tmem_ld16_nowait(tO + d, o[0]);
            tmem_ld16_nowait(tO + d + 16, o[1]);
            tmem_wait_ld();
            reg_fence(o[0]);
            reg_fence(o[1]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i >> 4][i & 15] = 0u;
        }
        auto val = [&](int i) { return __uint_as_float(o[i >> 4][i & 15]); };
        if constexpr (HALVES) {
            if (have && rows > (warp & 3) * 32) {
                float4 *at = box + (d & 32) / 4 * kRows + r;   // the box holds two rounds: what a round overwrites was read before the barrier of the last one
                if (st == 1)
#pragma unroll
                    for (int i = 0; i < 32; i += 4) at[(i / 4) * kRows] = make_float4(val(i), val(i + 1), val(i + 2), val(i + 3));
                if (d == 96) fence_proxy_async();   // the box is Q's memory again
                rows_sync();
                if (st == 0)
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 x = at[(i / 4) * kRows];
                        const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[(i + e) >> 4][(i + e) & 15] = __float_as_uint(val(i + e) * keep + y[e] * add);
                    }
                if (d == 96) fence_proxy_async();
            }
            if (st == 1) continue;
        }
        if (fix && mine) {
            for (int t = f0; t < f1; ++t) {
                if (TREE && !(nodes >> t & 1ull)) continue;
                const uint16_t *v = static_cast<const uint16_t *>(p.v.p) + (int64_t)((TREE ? pc.q0 : pc.k0) + t) * p.v.token +
                                    (int64_t)pc.g * p.v.head + d;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (not_finite<F16>(v[i]) & 0xFFFFu) o[i >> 4][i & 15] = __float_as_uint(val(i) + widen<F16>(v[i]));
            }
        }
        if (!whole) {
            if (mine) {
                float4 *part = p.part + (slot * 32 + d / 4) * p.rows_cap + in_tile;
#pragma unroll
                for (int i = 0; i < 32; i += 4) part[(i / 4) * p.rows_cap] = make_float4(val(i), val(i + 1), val(i + 2), val(i + 3));
            }
            continue;
        }
        // the row's 16-byte units are rotated by the row so that neither way meets a bank twice
        if (p.out_f32) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4 *>(line + (((i >> 2) ^ (lane & 7)) << 4)) =
                    make_float4(val(i) * inv, val(i + 1) * inv, val(i + 2) * inv, val(i + 3) * inv);
        } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
                *reinterpret_cast<uint4 *>(line + (((((d & 32) + i) >> 3) ^ (lane & 7)) << 4)) =
                    make_uint4(pack16<F16>(val(i) * inv, val(i + 1) * inv), pack16<F16>(val(i + 2) * inv, val(i + 3) * inv),
                               pack16<F16>(val(i + 4) * inv, val(i + 5) * inv), pack16<F16>(val(i + 6) * inv, val(i + 7) * inv));
            if ((d & 32) == 0) continue;
        }
        __syncwarp();   // eight lanes write a row's 128 bytes
        const int at = (d + 32) * unit - 128 + 16 * (lane & 7);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3), row = (warp & 3) * 32 + rr;
            const uint4 x = *reinterpret_cast<const uint4 *>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            if (row < rows) *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + output(row) * (128 * unit) + at) = x;
        }
    }
    __syncwarp();
    if (!mine || (HALVES && st == 1)) return;
    if (!whole) p.ml[slot * p.rows_cap + in_tile] = make_float2(m * p.scale_log2, l);
    else if (p.lse) p.lse[output(r)] = l == 0.0f ? -INFINITY : m * p.scale + logf(l);
}

// The next published piece (a warp); false when the wait ran out.  A reader gives it back with done().
struct Pieces {
    Ctrl &ct;
    int no = 0;   // pieces taken

    __device__ __forceinline__ bool next(volatile int *abort_flag, const Piece *&pc) {
        pc = &ct.pieces[no % kPieces];
        return wait_all(&ct.pfull[no % kPieces], (uint32_t)(no / kPieces) & 1u, abort_flag);
    }
    __device__ __forceinline__ void done() {   // lane 0, once the warp has read all it needs
        mbar_arrive(&ct.pempty[no++ % kPieces]);
    }
};

// HALVES: every tile has at most one stream's rows; both streams take them, each with half of a step's keys.
template <bool F16, bool TREE, bool HALVES, bool TILES>
__global__ void __launch_bounds__(kThreads, 1)
    dense_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kc,
                 const __grid_constant__ CUtensorMap tm_vc, const __grid_constant__ CUtensorMap tm_o,
                 const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem + kOffRing;
    Ctrl &ct = *reinterpret_cast<Ctrl *>(smem + kOffCtrl);
    volatile int *abort_flag = &ct.abort;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&ct.full[i], 1);
            mbar_init(&ct.empty[i], 2 + (i & 1));   // both streams, and for V (in the odd slots) warp 3
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ct.qfull[i], 1);
            mbar_init(&ct.qempty[i], HALVES && i == 1 ? 4 : 1);   // there, a warp of stream 0 each
            mbar_init(&ct.sfull[i], 1);
            for (int h = 0; h < 2; ++h) mbar_init(&ct.pready[i][h], 4);   // one arrival per warp of the stream
            mbar_init(&ct.ofull[i], 1);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&ct.pfull[i], 1);
            mbar_init(&ct.pempty[i], 11);  // every warp but the one that publishes
        }
        mbar_init(&ct.turn[0], 1);
        mbar_init(&ct.turn[1], 1);
        for (int i = 0; i < kSlots / 2; ++i) mbar_init(&ct.clean[i], 1);
        mbar_init(&ct.drain[0], 1);
        mbar_init(&ct.drain[1], 1);
        ct.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane < (TILES ? 6 : 5)) {
        const CUtensorMap *m = lane == 0 ? &tm_q : lane == 1 ? &tm_k : lane == 2 ? &tm_v : lane == 3 ? &tm_kc : lane == 4 ? &tm_vc : &tm_o;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    wait_prior_grid();   // nothing the caller wrote is read, and no tensor memory taken, before this
    allow_dependent_launch();
    if (warp == 1) {
        tmem_alloc(&ct.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)ct.tmem);

    int it = 0;                      // slots of the ring used so far
    uint32_t queries[2] = {0, 0};    // and Q tiles copied
    if (warp == 0) {
        // ---------------- pieces and copies: Q, K and V of each step, K first
        if (lane == 0) {
            p.desc[2 * (size_t)blockIdx.x] = make_int4(0, 0, 0, 0);
            p.desc[2 * (size_t)blockIdx.x + 1] = make_int4(0, 0, 0, 0);
        }
        Walk<TREE, HALVES> walk;
        find_share(p, ct, walk);
        if (lane == 0) ct.dealing = walk.rule == kDealt;
        Piece pc;
        int step = 0, no = 0;
        bool ok = true;
        const uint32_t qbytes = (uint32_t)(p.toks * p.group * 256);
        auto load_q = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!ok || pc.e[i] <= pc.s0) continue;
                if (!(ok = wait_all(&ct.qempty[i], (queries[i] & 1u) ^ 1u, abort_flag))) continue;
                ++queries[i];
                if (lane != 0) continue;
                uint8_t *to = smem + kOffQ + i * kQBytes;
                mbar_expect_tx(&ct.qfull[i], qbytes);
                const int row = pc.q0 + pc.tok0 + (HALVES ? 0 : i * p.toks);
                tma_load_3d(to, &tm_q, &ct.qfull[i], 0, pc.g * p.group, row);
                tma_load_3d(to + kQBytes / 2, &tm_q, &ct.qfull[i], 64, pc.g * p.group, row);
            }
        };
        while (ok) {
            const bool more = walk.next(p, ct, pc);
            pc.stop = !more;
            pc.bad = 0;
            if (!(ok = wait_all(&ct.pempty[no % kPieces], ((uint32_t)(no / kPieces) & 1u) ^ 1u, abort_flag))) break;
            if (lane == 0) {
                ct.pieces[no % kPieces] = pc;
                mbar_arrive(&ct.pfull[no % kPieces]);
            }
            ++no;
            if (!more) break;
            int pages = 0, ahead = 0;   // 32 entries of the table, a lane each, and the 32 after them
            const int nb = TREE ? (pc.lk + 63) >> 6 : 0;
            auto entries = [&](int chunk) {
                const int i = chunk * 32 + lane;
                return i < nb ? p.table[(size_t)pc.s * p.table_stride + i] : -1;
            };
            for (int j0 = pc.s0; ok && j0 < pc.s1; ++j0, ++step) {
                const int j = TREE ? j0 : step_at(j0, pc.s0, pc.s1, pc.first);
                const bool paged = TREE && j < pc.n - 1;
                int page[2] = {0, 0};
                if (paged) {
                    if (j == pc.s0) {
                        pages = entries(j >> 4);
                        ahead = entries((j >> 4) + 1);
                    } else if ((j & 15) == 0) {
                        pages = ahead;
                        ahead = entries((j >> 4) + 1);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        page[h] = __shfl_sync(~0u, pages, 2 * (j & 15) + h);
                        int valid = min(max(pc.lk - j * kKeys - h * 64, 0), 64);
                        if (page[h] < 0 || page[h] >= p.n_pages) {
                            if (valid > 0 && lane == 0) atomicOr(p.flags, QSA_FLAG_BAD_ID);
                            page[h] = p.n_kv * p.n_pages;   // behind the pool: the copy fills in zeros
                            valid = 0;
                        } else {
                            page[h] += pc.g * p.n_pages;
                        }
                        if (lane == 0) (h ? ct.info[step % kInfo].y : ct.info[step % kInfo].x) = valid;
                    }
                }
                for (int kv = 0; kv < 2; ++kv, ++it) {
                    const int slot = it % kSlots;
                    if (!(ok = wait_all(&ct.empty[slot], ((uint32_t)(it / kSlots) & 1u) ^ 1u, abort_flag))) break;
                    if (lane == 0) {
                        uint8_t *to = ring + slot * kSlotBytes;
                        uint64_t *bar = &ct.full[slot];
                        mbar_expect_tx(bar, kSlotBytes);
                        if (!paged) {
                            const int row = TREE ? pc.q0 : pc.k0 + j * kKeys;
                            const CUtensorMap *m = kv ? &tm_v : &tm_k;
                            tma_load_3d(to, m, bar, 0, row, pc.g);
                            tma_load_3d(to + kSlotBytes / 2, m, bar, 64, row, pc.g);
                        } else if (kv == 0) {   // two halves of 64 dimensions, each 128 token rows
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int row = page[h] * 64;
                                tma_load_2d(to + h * 8192, &tm_kc, bar, 0, row);
                                tma_load_2d(to + kSlotBytes / 2 + h * 8192, &tm_kc, bar, 64, row);
                            }
                        } else {                // two pages of 128 dimension rows
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                tma_load_2d(to + h * 16384, &tm_vc, bar, 0, page[h] * 128);
                        }
                    }
                    if (kv == 0 && j0 == pc.s0) load_q();   // behind the first K: the last piece may still read Q
                    if (!ok) {
                        ++it;
                        break;
                    }
                }
            }
            if (lane == 0 && ok) describe(p, pc);
        }
    } else if (warp == 1 || warp == 2) {
        // ---------------- products of a stream, issued by one lane.  The streams take turns (a stream's 16 MMAs of a step
        // run back to back while the other one's softmax does), and each waits for all it needs before its turn, so that
        // its waits lie behind the other one's products.  An MMA takes 47 cycles to issue and 64 to form: one warp alone, with
        // the waits between, issues both streams' more slowly than the tensor cores form them.
        const int st = warp - 1;
        constexpr uint32_t kDescS = idesc(F16 ? 0 : 1, kRows, HALVES ? 64 : 128), kDesc = idesc(F16 ? 0 : 1, kRows, 128);
        constexpr int kSteps = HALVES ? 4 : 8;   // of 16 keys
        const uint32_t smem0 = (uint32_t)uniform((int)smem_u32(smem));
        const uint64_t q_desc = sdesc(smem0 + kOffQ + st * kQBytes), k_desc = sdesc(smem0 + kOffRing);
        const uint64_t v_desc = sdesc_mn128(smem0 + kOffRing, 16384);
        const uint32_t tS = tmem + kColS + st * 128, tO = tmem + kColO + st * 128;
        uint32_t nq = 0, np = 0, cleaned = 0, turns = 0;
        bool ok = true;
        Pieces pieces{ct};
        const Piece *pp;
        auto slot_full = [&](int i) { return wait_all(&ct.full[i % kSlots], (uint32_t)(i / kSlots) & 1u, abort_flag); };
        auto my_turn = [&]() { return wait_all(&ct.turn[st], (turns++ & 1u) ^ (st == 0 ? 1u : 0u), abort_flag); };
        auto logits = [&](int kit, bool last) {   // one lane
            const uint64_t b = k_desc + (uint64_t)((kit % kSlots) * (kSlotBytes >> 4) + (HALVES ? st * 512 : 0));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int off = (k >> 2) * 1024 + (k & 3) * 2;
                mma<MmaKind::f16>(tS, q_desc + off, b + off, kDescS, k > 0);
            }
            mma_commit(&ct.sfull[st]);
            mma_commit(&ct.empty[kit % kSlots]);
            if (last && !(HALVES && st == 1)) mma_commit(&ct.qempty[st]);   // there, Q's memory is used once more
        };
        while (ok) {
            if (!(ok = pieces.next(abort_flag, pp)) || pp->stop) break;
            // a stream that is done with its steps still takes its turns and gives the other one's slots back
            const int s0 = uniform(pp->s0), s1 = uniform(pp->s1), e = uniform(pp->e[st]), n = uniform(pp->n), lk = uniform(pp->lk),
                      first = uniform(pp->first);
            const int low = TREE ? lk : uniform(Seq<TREE>::keys_of(pp->lq, lk, pp->tok0));
            if (s1 > s0) {
                ok = slot_full(it) && (e <= s0 || wait_all(&ct.qfull[st], nq++ & 1u, abort_flag)) && my_turn();
                if (ok) {
                    tc_fence_after();
                    if (elect_one()) {
                        if (e > s0) logits(it, e == s0 + 1);
                        else mbar_arrive(&ct.empty[it % kSlots]);
                        mbar_arrive(&ct.turn[st ^ 1]);
                    }
                    __syncwarp();
                }
            }
            for (int j = s0; ok && j < s1; ++j, it += 2) {
                const int vslot = (it + 1) % kSlots;
                const bool paged = TREE && j < n - 1, more = j + 1 < s1;
                if (!(ok = slot_full(it + 1))) break;
                if (((TREE ? j : step_at(j, s0, s1, first)) + 1) * kKeys > low || (TREE && !paged)) {
                    const int i = vslot >> 1;   // warp 3 clears what must not be read
                    if (!(ok = wait_all(&ct.clean[i], cleaned >> i & 1u, abort_flag))) break;
                    cleaned ^= 1u << i;
                }
                if (!(ok = (!more || slot_full(it + 2)) && (j >= e || wait_all(&ct.pready[st][0], np & 1u, abort_flag)) && my_turn()))
                    break;
                tc_fence_after();
                if (j < e) {   // the weights come in two parts: the first one's products run while the second is formed
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == 1) {
                            if (!(ok = wait_all(&ct.pready[st][1], np++ & 1u, abort_flag))) break;
                            tc_fence_after();
                        }
                        if (elect_one()) {
                            if (paged) {
                                const uint64_t b = k_desc + (uint64_t)(vslot * (kSlotBytes >> 4) + (HALVES ? st * 1024 : 0));
#pragma unroll
                                for (int k = h * kSteps / 2; k < (h + 1) * kSteps / 2; ++k)
                                    mma_f16_ta(tO, tS + 8 * k, b + (k >> 2) * 1024 + (k & 3) * 2, kDesc, k > 0 || j > s0);
                            } else {
                                const uint64_t b = v_desc + (uint64_t)(vslot * (kSlotBytes >> 4) + (HALVES ? st * 512 : 0));
#pragma unroll
                                for (int k = h * kSteps / 2; k < (h + 1) * kSteps / 2; ++k)
                                    mma_f16_ta(tO, tS + 8 * k, b + k * 128, kDesc | kIdescBMn, k > 0 || j > s0);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
                if (elect_one()) {
                    if (j < e) {
                        if (j + 1 == e) mma_commit(&ct.ofull[st]);
                        mma_commit(&ct.empty[vslot]);
                    } else {
                        mbar_arrive(&ct.empty[vslot]);
                    }
                    if (j + 1 < e) logits(it + 2, e == j + 2);
                    else if (more) mbar_arrive(&ct.empty[(it + 2) % kSlots]);
                    mbar_arrive(&ct.turn[st ^ 1]);
                }
                __syncwarp();
            }
            if (lane == 0) pieces.done();
            else ++pieces.no;
        }
    } else if (warp == 3) {
        // ---------------- values at places that not every row sees: cleared before the product reads them
        Pieces pieces{ct};
        const Piece *pp;
        bool ok = true;
        int base = 0;
        while (ok) {
            if (!(ok = pieces.next(abort_flag, pp)) || pp->stop) break;
            const int s0 = pp->s0, s1 = pp->s1, n = pp->n, lq = pp->lq, lk = pp->lk, first = pp->first;
            const int low = TREE ? 0 : Seq<TREE>::keys_of(lq, lk, pp->tok0);
            const int high = TREE ? lq : Seq<TREE>::keys_of(lq, lk, min(pp->tok0 + p.tile, lq) - 1);
            for (int j0 = s0; ok && j0 < s1; ++j0) {
                const int j = TREE ? j0 : step_at(j0, s0, s1, first);
                const bool paged = TREE && j < n - 1;
                const int vit = base + 2 * (j0 - s0) + 1, vslot = vit % kSlots;
                if (!(ok = wait_all(&ct.full[vslot], (uint32_t)(vit / kSlots) & 1u, abort_flag))) break;
                // only a run's last steps hold such places
                if (TREE ? paged && (j + 1) * kKeys <= lk : (j + 1) * kKeys <= low) {
                    if (lane == 0) mbar_arrive(&ct.empty[vslot]);
                    continue;
                }
                uint8_t *v = ring + vslot * kSlotBytes;
                bool bad = false;
#pragma unroll 1
                for (int r = lane; r < kKeys; r += 32) {
                    if (!paged) {   // a token
                        const int t = TREE ? r : j * kKeys + r;
                        uint8_t *row = v + r * 128;
                        if (t >= high) {
#pragma unroll
                            for (int ch = 0; ch < 16; ++ch)
                                *reinterpret_cast<uint4 *>(row + (ch >> 3) * 16384 + ((ch & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                        } else if (t >= low) {   // seen by some of the rows
                            uint32_t acc[2] = {0u, 0u};
#pragma unroll
                            for (int ch = 0; ch < 16; ++ch) {   // in any order: the swizzle moves units within the row
                                const uint4 x = *reinterpret_cast<const uint4 *>(row + (ch >> 3) * 16384 + (((ch ^ r) & 7) << 4));
                                acc[0] = probe<F16>(x.x, acc[0]);
                                acc[1] = probe<F16>(x.y, acc[1]);
                                acc[0] = probe<F16>(x.z, acc[0]);
                                acc[1] = probe<F16>(x.w, acc[1]);
                            }
                            if (not_finite<F16>(acc[0]) | not_finite<F16>(acc[1])) {
                                bad = true;
#pragma unroll 1
                                for (int e = 0; e < 64; ++e) {
                                    uint32_t *x = reinterpret_cast<uint32_t *>(row + (e >> 5) * 16384) + (e & 31);
                                    *x &= ~not_finite<F16>(*x);
                                }
                            }
                        }
                    } else {        // a dimension: every row sees the tokens that are there
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int valid = min(max(lk - j * kKeys - 64 * h, 0), 64);
                            for (int ch = valid >> 3; ch < 8; ++ch) {
                                uint8_t *x = v + h * 16384 + r * 128 + ((ch ^ (r & 7)) << 4);
                                if (8 * ch >= valid) {
                                    *reinterpret_cast<uint4 *>(x) = make_uint4(0u, 0u, 0u, 0u);
                                } else {
                                    uint16_t *e = reinterpret_cast<uint16_t *>(x);
                                    for (int t = valid - 8 * ch; t < 8; ++t) e[t] = 0;
                                }
                            }
                        }
                    }
                }
                if (bad) ct.pieces[pieces.no % kPieces].bad = 1;
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ct.clean[vslot >> 1]);
                    mbar_arrive(&ct.empty[vslot]);
                }
            }
            base += 2 * (s1 - s0);
            __syncwarp();
            if (lane == 0) pieces.done();
            else ++pieces.no;
        }
    } else {
        // ---------------- softmax and epilogue of a stream, a thread a row
        const int st = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + kColS + st * 128, tO = tmem + lanes + kColO + st * 128;
        const int first_tok = HALVES ? 0 : st * p.toks;                     // of the stream, in a tile
        const int my_tok = first_tok + (int)(r * p.by_group >> 16);        // this row's
        constexpr int kCols = HALVES ? 64 : 128;                           // keys of a stream in a step
        Pieces pieces{ct};
        const Piece *pp;
        int step0 = 0;
        uint32_t ns = 0, no = 0;
        bool ok = true;
        // HALVES: the streams meet at named barriers, which know no limit, so no warp may leave alone: one whose wait ran
        // out goes on without waiting, and all leave together before the next piece.
        while (true) {
            ok = pieces.next(abort_flag, pp) && ok;
            if ((HALVES ? any_of(3, 256, !ok) : !ok) || pp->stop) break;
            const int n = TREE ? pp->n : 0;
            // what this row sees
            int low = 0;                                // prompts: keys of the stream's first row
            unsigned long long nodes = 0ull;            // trees: of the drafts
            if constexpr (TREE) {
                if (pp->e[st] == n && n > pp->s0) nodes = ancestors(p, pp->q0, pp->lq, min(pp->tok0 + my_tok, pp->lq - 1));
            } else {
                low = Seq<TREE>::keys_of(pp->lq, pp->lk, min(pp->tok0 + first_tok, pp->lq - 1));
            }
            // Prompts: keys that this row sees.  What only half-seen steps and the end need is taken from the piece again there: the
            // steps that are seen whole fill the registers (16,384 tokens 2.43 -> 2.32 ms).
            auto limit = [&]() { return Seq<TREE>::keys_of(pp->lq, pp->lk, pp->tok0 + my_tok); };
            float m = -INFINITY, l = 0.0f;
            int place = step0, j = TREE ? pp->s0 : pp->first;   // the step's place among all of the CTA's, and the step
#pragma unroll 1
            for (int left = pp->e[st] - pp->s0; left > 0; --left, ++place, j = TREE || j + 1 < pp->s1 ? j + 1 : pp->s0) {
                ok = ok && wait_all(&ct.sfull[st], ns++ & 1u, abort_flag);
                if (!HALVES && !ok) break;
                tc_fence_after();
                // which keys this row sees, 32 a word; all of them in most steps
                const bool paged = TREE && j < n - 1;
                int valid[2] = {0, 0};
                if (paged) {
                    const int2 x = ct.info[place % kInfo];
                    valid[0] = x.x;
                    valid[1] = x.y;
                }
                const bool some = TREE ? (HALVES ? valid[st] : min(valid[0], valid[1])) < 64 : (j + 1) * kKeys > low;
                int lim = 0;
                auto sees = [&](int q) -> uint32_t {
                    const int at = (HALVES ? 64 * st : 0) + 32 * q;   // the word's first key in the step
                    if (TREE && !paged) return at == 0 ? (uint32_t)nodes : at == 32 ? (uint32_t)(nodes >> 32) : 0u;
                    const int left = TREE ? valid[at >> 6] - (at & 63) : lim - j * kKeys - at;
                    return left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u;
                };
                // the row's reference, given the step's largest logit
                auto settle = [&](float now) {
                    const bool risen = (now - m) * p.scale_log2 > kRise;   // from nothing seen, by anything
                    if (!__any_sync(~0u, risen && m > -INFINITY)) {        // O is not there yet, or 0, where nothing was seen
                        if (risen) m = now;
                        return;
                    }
                    // S of this step is complete, so every product before it is: O may be scaled in place
                    const float f = risen ? ex2((m - now) * p.scale_log2) : 1.0f;
                    if (risen) m = now;
                    l *= f;
#pragma unroll 1
                    for (int d = 0; d < 128; d += 16) {
                        uint32_t o[16];
                        tmem_ld16_nowait(tO + d, o);
                        tmem_wait_ld();
                        reg_fence(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st16(tO + d, o);
                    }
                };
                f32x2 sum[2] = {pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
                auto weigh = [&](float s0, float s1, f32x2 c2, f32x2 nm2, int i) -> uint32_t {
                    float y0, y1;
                    unpack2(fma2(pack2(s0, s1), c2, nm2), y0, y1);
                    y0 = ex2(y0);
                    y1 = ex2(y1);
                    sum[i & 1] = add2(sum[i & 1], pack2(y0, y1));
                    return pack16<F16>(y0, y1);
                };
                auto pass_on = [&](int h) {   // a part of the weights goes on as soon as it is there
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ct.pready[st][h]);
                };
                if (!some) {
                    uint32_t v[kCols / 16][16];
#pragma unroll
                    for (int h = 0; h < kCols / 64; ++h) tmem_ld64_nowait(tS + 64 * h, reinterpret_cast<uint32_t(&)[4][16]>(v[4 * h]));
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < kCols / 16; ++i) reg_fence(v[i]);
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < kCols; i += 2)
                        top[(i >> 1) & 3] = fmaxf(top[(i >> 1) & 3], fmaxf(__uint_as_float(v[i >> 4][i & 15]),
                                                                           __uint_as_float(v[i >> 4][(i & 15) + 1])));
                    settle(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
                    const float c = p.scale_log2, mc = m == -INFINITY ? 0.0f : m * c;
                    const f32x2 c2 = pack2(c, c), nm2 = pack2(-mc, -mc);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int q = 0; q < kCols / 64; ++q) {   // 32 keys
#pragma unroll
                            for (int i = 0; i < 16; ++i) {   // in place: pair i over value i
                                const int k = h * (kCols / 2) + 32 * q + 2 * i, to = h * (kCols / 2) + 32 * q + i;
                                v[to >> 4][to & 15] = weigh(__uint_as_float(v[k >> 4][k & 15]), __uint_as_float(v[k >> 4][(k & 15) + 1]), c2, nm2, i);
                            }
                            tmem_st16(tS + h * (kCols / 4) + 16 * q, v[(h * (kCols / 2) + 32 * q) >> 4]);
                        }
                        pass_on(h);
                    }
                } else {
                    // 32 keys a round, read twice, in little code: short runs spend their time in steps like this one, and on
                    // fetching instructions
                    if constexpr (!TREE) lim = limit();
                    auto logits_of = [&](int q, uint32_t (&x)[2][16]) {
                        tmem_ld16_nowait(tS + 32 * q, x[0]);
                        tmem_ld16_nowait(tS + 32 * q + 16, x[1]);
                        const uint32_t word = sees(q);
                        tmem_wait_ld();
                        reg_fence(x[0]);
                        reg_fence(x[1]);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(word & 1u << i)) x[i >> 4][i & 15] = 0xFF800000u;
                    };
                    float now = -INFINITY;
#pragma unroll 1
                    for (int q = 0; q < kCols / 32; ++q) {
                        uint32_t x[2][16];
                        logits_of(q, x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) now = fmaxf(now, fmaxf(__uint_as_float(x[0][i]), __uint_as_float(x[1][i])));
                    }
                    settle(now);
                    const float c = p.scale_log2, mc = m == -INFINITY ? 0.0f : m * c;
                    const f32x2 c2 = pack2(c, c), nm2 = pack2(-mc, -mc);
#pragma unroll 1
                    for (int q = 0; q < kCols / 32; ++q) {
                        uint32_t x[2][16], w[16];
                        logits_of(q, x);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = weigh(__uint_as_float(x[i >> 3][2 * (i & 7)]), __uint_as_float(x[i >> 3][2 * (i & 7) + 1]), c2, nm2, i);
                        tmem_st16(tS + 16 * q, w);   // over logits that have been read
                        if (q == kCols / 64 - 1) pass_on(0);
                    }
                    pass_on(1);
                }
                float a, b;
                unpack2(add2(sum[0], sum[1]), a, b);
                l += a + b;
            }
            if (!HALVES && !ok) break;
            const int rows = pp->rows[st];
            const bool have = pp->e[st] > pp->s0;
            if (HALVES || rows > (warp & 3) * 32 || have) {
                if (have) {
                    ok = ok && wait_all(&ct.ofull[st], no++ & 1u, abort_flag);
                    if (!HALVES && !ok) break;
                    tc_fence_after();
                }
                finish<F16, TREE, HALVES, TILES>(p, ct, *pp, have, tO, smem + kOffStage + (warp - 4) * kStageBytes,
                                          reinterpret_cast<float4 *>(smem + kOffQ + kQBytes), m, l, TREE ? 0 : limit(), nodes, rows, &tm_o);
                tc_fence_before();
                if (HALVES && st == 0 && have) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ct.qempty[1]);
                }
            }
            step0 += pp->s1 - pp->s0;
            __syncwarp();
            if (lane == 0) pieces.done();
            else ++pieces.no;
        }
        if (TILES) bulk_wait();
        tc_fence_before();
    }
    __syncthreads();
    if (ct.abort && lane == 0) {   // copies and products in flight end before their memory goes
        if (warp == 0) {
            for (int i = max(0, it - kSlots); i < it; ++i) mbar_drain(&ct.full[i % kSlots], (uint32_t)(i / kSlots) & 1u);
            for (int i = 0; i < 2; ++i)
                if (queries[i] > 0) mbar_drain(&ct.qfull[i], (queries[i] - 1u) & 1u);
        }
        if (warp == 1 || warp == 2) {
            mma_commit(&ct.drain[warp - 1]);
            mbar_drain(&ct.drain[warp - 1], 0);
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0) {
        if (ct.abort) atomicOr(p.flags, QSA_FLAG_WAIT_TIMEOUT);
        if (ct.dealing) {   // the last CTA leaves the counts at 0
            unsigned *dealt = p.dealt + 2 * (blockIdx.x % (unsigned)p.row_tiles);
            if (atomicAdd(dealt + 1, 1u) + 1u == (unsigned)p.shares) dealt[0] = dealt[1] = 0u;
        }
    }
}

// Runs that several CTAs worked on: a CTA per (share that a run begins in and does not end in, 32 rows), a lane per row.
// The partials O_c of the shares from there to the run's end are weighted 2^(m_c - M).
constexpr int kJoinWarps = 8;
constexpr int kJoinDims = 4;   // groups of four dimensions that a CTA joins where parts may be many,
constexpr int kJoinGroups = 2; // and that a warp joins where they are few (4 loads' time for 64 sequences 3 us more; 1, idle CTAs 2 us)
constexpr int kJoinTurns = (kMaxCtas + kJoinWarps - 1) / kJoinWarps;

// MANY: few rows (a decode step), so a run may lie in many parts: the warps share them out and meet in shared memory.
// Otherwise a warp takes eight dimensions of all parts.
template <bool F16, bool MANY>
__global__ void __launch_bounds__(32 * kJoinWarps) combine_kernel(const __grid_constant__ Params p, int grid) {
    wait_prior_grid();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, step = p.row_tiles;
    const int4 d = p.desc[2 * (size_t)blockIdx.x + 1];
    if (d.x == 0) return;
    const int in_tile = blockIdx.y * 32 + lane, st = blockIdx.y >> 2, r = in_tile & (kRows - 1);
    const int tok = (int)(r * p.by_group >> 16), token = st * p.toks + tok;
    const bool mine = tok < p.toks && token < d.w;
    if (!__any_sync(~0u, mine)) return;   // the same in every warp
    int parts = 0;   // shares behind this one that hold a part
    for (int c0 = 1;; c0 += 32) {
        const long long c = blockIdx.x + (long long)(c0 + lane) * step;
        const int kind = c < grid ? p.desc[2 * c].x : 1;
        const unsigned ends = __ballot_sync(~0u, kind != 2);
        if (ends) {
            parts = c0 + __ffs(ends) - 1;
            break;
        }
    }
    auto slot = [&](int i) { return 2 * ((size_t)blockIdx.x + (size_t)i * step) + (i == 0 ? 1 : 0); };
    auto sums_of = [&](int i) { return p.ml[slot(i) * p.rows_cap + in_tile]; };   // a sum of 0: saw nothing
    auto part_of = [&](int i, int d4) { return p.part[(slot(i) * 32 + d4) * p.rows_cap + in_tile]; };
    auto add = [](float4 &o, float f, const float4 &y) {
        o.x = fmaf(f, y.x, o.x);
        o.y = fmaf(f, y.y, o.y);
        o.z = fmaf(f, y.z, o.z);
        o.w = fmaf(f, y.w, o.w);
    };
    const size_t at = (size_t)(d.z + token) * p.n_heads + d.y * p.group + (r - tok * p.group);
    auto put = [&](const float4 &x, float inv, int d4) { store4<F16>(p, at * 128 + 4 * d4, x.x * inv, x.y * inv, x.z * inv, x.w * inv); };
    float M = -INFINITY, L = 0.0f;
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (MANY) {
        __shared__ float top[kJoinWarps][32], sums[kJoinWarps][32];
        __shared__ float4 joined[kJoinWarps][kJoinDims][32];
        float2 ml[kJoinTurns];
#pragma unroll
        for (int k = 0; k < kJoinTurns; ++k) {
            const int i = warp + k * kJoinWarps;
            ml[k] = mine && i <= parts ? sums_of(i) : make_float2(-INFINITY, 0.0f);
        }
#pragma unroll
        for (int k = 0; k < kJoinTurns; ++k)
            if (ml[k].y != 0.0f) M = fmaxf(M, ml[k].x);
        top[warp][lane] = M;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, top[w][lane]);
        float4 o[kJoinDims];
#pragma unroll
        for (int e = 0; e < kJoinDims; ++e) o[e] = zero;
#pragma unroll
        for (int k = 0; k < kJoinTurns; ++k) {
            const float f = ml[k].y == 0.0f ? 0.0f : ex2(ml[k].x - M);
            L = fmaf(f, ml[k].y, L);
            if (f == 0.0f) continue;
#pragma unroll
            for (int e = 0; e < kJoinDims; ++e) add(o[e], f, part_of(warp + k * kJoinWarps, blockIdx.z * kJoinDims + e));
        }
        sums[warp][lane] = L;
#pragma unroll
        for (int e = 0; e < kJoinDims; ++e) joined[warp][e][lane] = o[e];
        __syncthreads();
        if (warp >= kJoinDims || !mine) return;
        L = 0.0f;
        float4 x = zero;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            add(x, 1.0f, joined[w][warp][lane]);
            L += sums[w][lane];
        }
        put(x, L == 0.0f ? 0.0f : 1.0f / L, blockIdx.z * kJoinDims + warp);
    } else {
        if (!mine) return;
#pragma unroll 4
        for (int i = 0; i <= parts; ++i) {
            const float2 ml = sums_of(i);
            M = fmaxf(M, ml.y == 0.0f ? -INFINITY : ml.x);
        }
        constexpr int kDims = kJoinGroups;
        const int d0 = blockIdx.z * kJoinWarps * kDims + warp;
        float4 x[kDims];
#pragma unroll
        for (int e = 0; e < kDims; ++e) x[e] = zero;
#pragma unroll 4
        for (int i = 0; i <= parts; ++i) {
            const float2 ml = sums_of(i);
            float4 y[kDims];
#pragma unroll
            for (int e = 0; e < kDims; ++e) y[e] = part_of(i, d0 + e * kJoinWarps);
            const float f = ml.y == 0.0f ? 0.0f : ex2(ml.x - M);
            L = fmaf(f, ml.y, L);
#pragma unroll
            for (int e = 0; e < kDims; ++e)
                if (f != 0.0f) add(x[e], f, y[e]);
        }
#pragma unroll
        for (int e = 0; e < kDims; ++e) put(x[e], L == 0.0f ? 0.0f : 1.0f / L, d0 + e * kJoinWarps);
    }
    if (warp == 0 && blockIdx.z == 0 && p.lse) p.lse[at] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// Rows of a tile that `tokens` tokens can fill.
int rows_cap(int tokens, int group) {
    return tokens > kRows / group ? 2 * kRows : (tokens * group + 31) / 32 * 32;
}

template <bool F16, bool TREE, bool HALVES, bool TILES>
qsa_status launch_typed(const CUtensorMap (&m)[6], const Params &p, int grid, int most_steps, cudaStream_t s) {
    static std::mutex mu;
    static bool opted_in[64] = {false};
    int dev = 0;
    qsa_status st = check_cuda(cudaGetDevice(&dev), "cudaGetDevice");
    if (st != QSA_OK) return st;
    if (dev < 0 || dev >= 64) return fail(QSA_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!opted_in[dev]) {
            st = check_cuda(cudaFuncSetAttribute(dense_kernel<F16, TREE, HALVES, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem),
                            "cudaFuncSetAttribute(dense attention)");
            if (st != QSA_OK) return st;
            opted_in[dev] = true;
        }
    }
    st = launch_dependent("dense_kernel launch", dense_kernel<F16, TREE, HALVES, TILES>, grid, kThreads, kSmem, s, m[0], m[1], m[2],
                          m[3], m[4], m[5], p);
    if (st != QSA_OK || most_steps <= kWhole) return st;
    const long long runs = (long long)p.n_seqs * p.n_kv, parts = std::min<long long>(p.shares / runs, most_steps / kLeast);
    const bool many = p.rows_cap <= 64 && parts >= kManyParts;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)(p.rows_cap / 32), 32 / (many ? kJoinDims : kJoinWarps * kJoinGroups));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return check_cuda(many ? cudaLaunchKernelEx(&cfg, combine_kernel<F16, true>, p, grid)
                           : cudaLaunchKernelEx(&cfg, combine_kernel<F16, false>, p, grid),
                      "combine_kernel launch");
}

template <bool TREE>
qsa_status launch(const DenseArgs &a, cudaStream_t s) {
    Params p{};
    p.v = a.v;
    p.cu_q = a.cu_q;
    p.cu_k = a.cu_k;
    p.n_seqs = a.n_seqs;
    p.total_q = a.total_q;
    p.total_k = a.total_k;
    p.n_heads = a.n_heads;
    p.n_kv = a.n_kv_heads;
    p.group = a.n_heads / a.n_kv_heads;
    p.toks = kRows / p.group;
    // No tile holds a second stream's rows: both take the first's, half a step each (us, halves / whole steps: a query at 9,000
    // tokens 20.3 / 22.1, 16 decodes of 500 tokens 17.1 / 18.4, 258,000 tokens 94.5 / 94.7)
    const bool halves = (TREE ? a.max_nodes : a.total_q) <= p.toks;
    p.tile = halves ? p.toks : 2 * p.toks;
    const int most = TREE && a.max_nodes < a.total_q ? a.max_nodes : a.total_q;   // tokens of a sequence
    p.rows_cap = rows_cap(most, p.group);
    p.by_group = (65536u + (uint32_t)p.group - 1u) / (uint32_t)p.group;
    p.scale = a.scale;
    p.scale_log2 = a.scale < 2e38f ? a.scale * 1.4426950408889634f : 3e38f;
    p.out = a.out;
    p.out_f32 = a.out_dt == QSA_F32;
    p.lse = a.lse;
    p.parents = a.parents;
    p.max_nodes = a.max_nodes;
    p.table = a.table.table;
    p.table_stride = a.table.stride;
    p.max_pages = a.table.max_pages;
    p.n_pages = a.table.n_pages;
    p.n_tokens = a.n_tokens;
    p.flags = a.flags;
    p.dealt = static_cast<unsigned *>(a.ws) + 16;   // in the first 256 bytes, behind the flags word; two counts for each tile of rows
    char *ws = static_cast<char *>(a.ws) + 256;
    p.desc = reinterpret_cast<int4 *>(ws);
    p.ml = reinterpret_cast<float2 *>(ws + kMaxCtas * 2 * sizeof(int4));
    p.part = reinterpret_cast<float4 *>(ws + kMaxCtas * 2 * (sizeof(int4) + (size_t)p.rows_cap * sizeof(float2)));
    const int ctas = num_sms() < kMaxCtas ? num_sms() : kMaxCtas;
    p.row_tiles = TREE ? (a.max_nodes + p.tile - 1) / p.tile : 1;
    p.shares = ctas / p.row_tiles;
    const int grid = p.shares * p.row_tiles;
    // of a run, as far as the sizes tell
    const int most_steps = ((TREE ? 64 * a.table.max_pages : a.total_k) + kKeys - 1) / kKeys + (TREE ? 1 : 0);
    CUtensorMap m[6];
    const Rows16 &k = a.total_k > 0 ? a.k : a.q, &v = a.total_k > 0 ? a.v : a.q;   // without keys nothing is loaded
    const int rows = a.total_k > 0 ? a.total_k : 1, heads = a.total_k > 0 ? a.n_kv_heads : 1;
    qsa_status st;
    if ((st = get_rows_map(&m[0], a.q, a.total_q, a.n_heads, true, p.toks, p.group)) != QSA_OK ||
        (st = get_rows_map(&m[1], k, rows, heads, false, kKeys, 1)) != QSA_OK ||
        (st = get_rows_map(&m[2], v, rows, heads, false, kKeys, 1)) != QSA_OK)
        return st;
    m[3] = m[1];
    m[4] = m[2];
    m[5] = m[0];
    if (TREE) {
        const uint64_t pages = (uint64_t)a.n_kv_heads * a.table.n_pages;
        if ((st = get_map(&m[3], a.kcache, 2, 128, pages * 64, 64)) != QSA_OK ||
            (st = get_map(&m[4], a.vcache_t, 2, 64, pages * 128, 128)) != QSA_OK)
            return st;
    }
    const bool f16 = a.dt == QSA_F16;
    if (halves)
        return f16 ? launch_typed<true, TREE, true, false>(m, p, grid, most_steps, s)
                   : launch_typed<false, TREE, true, false>(m, p, grid, most_steps, s);
    if constexpr (!TREE) {
        // 16-bit rows of whole tokens a warp may leave by TMA: the lanes that read the stage back and store it take issue slots that the
        // other warps need, but the branch costs the steps registers (us, by TMA / not: 20 prompts of 300 tokens 75 / 86, one of
        // 1,024 25.8 / 26.6, 8 of 2,000 370 / 377, one of 4,096 170 / 168.5, of 8,192 602 / 587, 256 queries behind 130,816 591 / 575)
        if (!p.out_f32 && 32 % p.group == 0 && a.total_k <= kShortKeys * (long long)a.n_seqs) {
            const Rows16 out{a.out, (int64_t)a.n_heads * 128, 128};
            if ((st = get_rows_map(&m[5], out, a.total_q, a.n_heads, true, 32 / p.group, p.group, 32)) != QSA_OK) return st;
            return f16 ? launch_typed<true, false, false, true>(m, p, grid, most_steps, s)
                       : launch_typed<false, false, false, true>(m, p, grid, most_steps, s);
        }
    }
    return f16 ? launch_typed<true, TREE, false, false>(m, p, grid, most_steps, s)
               : launch_typed<false, TREE, false, false>(m, p, grid, most_steps, s);
}

}  // namespace

size_t attention_ws_bytes(int rows, int n_heads, int n_kv_heads) {
    const int cap = rows_cap(rows, n_heads / n_kv_heads);
    return 256 + (size_t)kMaxCtas * 2 * (sizeof(int4) + (size_t)cap * (sizeof(float2) + 32 * sizeof(float4)));
}
qsa_status launch_prompt_attention(const DenseArgs &a, cudaStream_t s) { return launch<false>(a, s); }
qsa_status launch_tree_attention(const DenseArgs &a, cudaStream_t s) { return launch<true>(a, s); }

}  // namespace qsa
