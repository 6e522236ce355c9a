// qcache.cu -- writing token rows into the 4-bit KV cache and reading them back.
//
// A row x of 128 values is held as 16 levels between its minimum and its maximum:
//   scale = the least 16-bit value >= (max - min) / 15,
//   code  = (x - min) / scale, rounded half to even,   value = scale * code + min.
// Rounding the scale up keeps code <= 15 and |value - x| <= scale / 2 for every x; the
// minimum is one of the row's values, so it is exact.
//
// One CTA (256 threads) per (KV head, block of 64 tokens), four threads per token: thread
// c of a token holds its 16-byte units c, c + 4, c + 8 and c + 12 (8 dimensions each), so the
// four threads' accesses are neighbours, and units 8 apart are the low and the high nibbles
// of the same 8 bytes of K, which go from registers to the cache.  V is stored
// dimension-major: its codes pass through shared memory as bytes, are transposed four by four
// with byte permutes and exchanged among four lanes, and leave as whole 16-byte rows.  In a
// partial block only the call's own nibbles change, by an atomic exclusive-or of each word that
// holds others too, so that two appends may fill one block at the same time.
//
// Measured, 131,072 tokens x 4 KV heads, bf16: the reader moves its 340 MB in 52 us (6.5 TB/s, near
// the copy rate); the writer's 340 MB take 76 us: it issues 0.70 instructions a cycle and scheduler (15
// a value, half of them the quotient and its rounding), against 50 us at the copy rate.  Units dealt as
// 32 consecutive bytes per thread instead of one 16-byte unit in four took 65 us (reader);
// codes by divisions and byte-wise transposes 203 us (writer).
#include <cfloat>

#include "qcache.cuh"
#include "qsa_device.cuh"

namespace qsa {
namespace {

constexpr int kNT = 256;
constexpr float kNearHalf = 0.5f - 0x1p-18f;   // a quotient may be 2^-21 off
constexpr int kPitch = 136;   // bytes per token of the staged V codes: rows four apart start 8 banks apart

struct RowPtr {
    const uint8_t *p;
    int64_t token_bytes, head_bytes;
};
struct RowPtrW {
    uint8_t *p;
    int64_t token_bytes, head_bytes;
};

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// (x - lo) / scale rounded half to even, exactly: the difference as an unevaluated sum
// a + e, a first quotient (at most one off), and the sign of the remainder against
// half a step.  Each fp32 step before the last comparison is exact (a + e is the two-sum of O. Moller and
// D. E. Knuth).
__device__ __forceinline__ int exact_code(float x, float lo, float scale) {
    const float a = x - lo;
    const float bb = a - x;
    const float e = (x - (a - bb)) + (-lo - bb);
    float c = rintf(__fdiv_rn(a, scale));
    const float r = fmaf(-c, scale, a);
    const float h = 0.5f * scale;
    const bool odd = ((int)c & 1) != 0;
    const float over = (r - h) + e, under = (r + h) + e;
    if (over > 0.0f || (over == 0.0f && odd)) c += 1.0f;
    else if (under < 0.0f || (under == 0.0f && odd)) c -= 1.0f;
    return min(max((int)c, 0), 15);
}

// One thread's 32 values of a row as 16 pairs: its units c, c + 4, c + 8, c + 12.
__device__ __forceinline__ void load_row(const uint8_t *row, int c, uint32_t (&x)[16]) {
    const uint4 *r = reinterpret_cast<const uint4 *>(row);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 a = r[c + 4 * i];
        x[4 * i] = a.x;
        x[4 * i + 1] = a.y;
        x[4 * i + 2] = a.z;
        x[4 * i + 3] = a.w;
    }
}

// Those units' codes by the exact comparison, from the row itself.  Rare, and out of line: it takes no registers
// from the common path.
template <bool F16>
__device__ __noinline__ uint4 exact_row(const uint8_t *row, int c, float lo, float scale) {
    uint32_t word[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            const uint16_t *x = reinterpret_cast<const uint16_t *>(row) + 8 * (c + (w < 2 ? 0 : 4)) + 4 * (w & 1) + j;
            const int c0 = exact_code(QFmt<F16>::lo(x[0]), lo, scale), c1 = exact_code(QFmt<F16>::lo(x[64]), lo, scale);
            word[w] |= (uint32_t)(c0 | (c1 << 4)) << (8 * j);
        }
    return make_uint4(word[0], word[1], word[2], word[3]);
}

// The row's codes (a nibble pair per byte: words 0 and 1 units c low and c + 8 high, words 2 and 3 units
// c + 4 and c + 12) and its (scale, minimum) pair; the four threads of a token call it together.
//
// The quotient (x - min) / scale comes from the reciprocal and one correction by its remainder (P. Markstein, IBM
// Journal of Research and Development 34, 1990), to half an fp32 step (2^-21 below 16).  Where x
// is 0 or at least kShort times the scale (and the minimum too), 2 (x - min) - (2n + 1) scale is a
// multiple of 2^-20 of the scale, so a quotient is a half exactly when its value is, and the
// rounding of the quotient is the exact one's; a row with a shorter x looks whether such an x has
// its quotient near a half, and only then takes the exact comparison.
template <bool F16>
__device__ __forceinline__ uint32_t quantise(const uint32_t (&x)[16], const uint8_t *row, int c, uint32_t (&packed)[4]) {
    using Fmt = QFmt<F16>;
    uint32_t mn2 = x[0], mx2 = x[0], ab2 = x[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
        mn2 = Fmt::min2(mn2, x[i]);
        mx2 = Fmt::max2(mx2, x[i]);
        ab2 = Fmt::min2(ab2, x[i] & 0x7FFF7FFFu);
    }
    float lo = min_nan(Fmt::lo(mn2), Fmt::hi(mn2)), hi = max_nan(Fmt::lo(mx2), Fmt::hi(mx2));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(kFull, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(kFull, hi, o));
    }
    lo = __fadd_rn(lo, 0.0f);   // -0 is held as +0
    // upward at every step: the least 16-bit value >= the exact (max - min) / 15 (15 times a
    // 16-bit value is an fp32 value, so no rounding passes one)
    const float range = __fsub_ru(hi, lo);
    if (!(range <= FLT_MAX)) {   // an infinity, a NaN or too wide: the row reads as NaN
        packed[0] = packed[1] = packed[2] = packed[3] = 0u;
        return F16 ? 0x7E007E00u : 0x7FC07FC0u;
    }
    const uint32_t sbits = Fmt::bits_up(__fdiv_ru(range, 15.0f));
    const float scale = Fmt::lo(sbits);
    bool exact = scale > 0.0f && scale < 1e-30f;   // no finite reciprocal, or a subnormal remainder
    const float inv = scale < 1e-30f ? 0.0f : __frcp_rn(scale);
    const float magic = 12582912.0f;               // 1.5 2^23: adding it rounds to an integer, half to even
    const f32x2 nlo2 = pack2(-lo, -lo), inv2 = pack2(inv, inv), nscale2 = pack2(-scale, -scale);
    const f32x2 magic2 = pack2(magic, magic), nmagic2 = pack2(-magic, -magic), sixteen2 = pack2(16.0f, 16.0f);
    auto quotients = [&](uint32_t pair) {
        const f32x2 d = add2(pack2(Fmt::lo(pair), Fmt::hi(pair)), nlo2), q0 = mul2(d, inv2);
        return fma2(fma2(q0, nscale2, d), inv2, q0);
    };
    const float least = scale * Fmt::kShort;
    const bool lo_short = fabsf(lo) < least;
    if (fminf(Fmt::lo(ab2), Fmt::hi(ab2)) < least || lo_short) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const f32x2 q = quotients(x[i]);
            float f0, f1;
            unpack2(fma2(add2(add2(q, magic2), nmagic2), pack2(-1.0f, -1.0f), q), f0, f1);
            exact |= fabsf(f0) > kNearHalf && (lo_short || fabsf(Fmt::lo(x[i])) < least);
            exact |= fabsf(f1) > kNearHalf && (lo_short || fabsf(Fmt::hi(x[i])) < least);
        }
        exact = exact && scale > 0.0f;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t byte[4];   // in the low bits of magic + low code + 16 x high code
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f32x2 t0 = add2(quotients(x[2 * w + j]), magic2);
            const f32x2 t1 = add2(add2(quotients(x[8 + 2 * w + j]), magic2), nmagic2);
            float b0, b1;
            unpack2(fma2(t1, sixteen2, t0), b0, b1);
            byte[2 * j] = __float_as_uint(b0);
            byte[2 * j + 1] = __float_as_uint(b1);
        }
        packed[w] = __byte_perm(__byte_perm(byte[0], byte[1], 0x0040), __byte_perm(byte[2], byte[3], 0x0040), 0x5410);
    }
    if (exact) {
        const uint4 all = exact_row<F16>(row, c, lo, scale);
        packed[0] = all.x;
        packed[1] = all.y;
        packed[2] = all.z;
        packed[3] = all.w;
    }
    return sbits | (Fmt::bits(lo) << 16);
}

// Words w[i] of four neighbouring lanes (q = lane & 3) as a 4 x 4 matrix, transposed: lane q gets word q of each.
__device__ __forceinline__ void transpose_lanes(uint32_t (&w)[4], int q) {
#pragma unroll
    for (int step = 1; step < 4; step <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & step) continue;
            const bool up = (q & step) != 0;
            const uint32_t got = __shfl_xor_sync(kFull, up ? w[i] : w[i + step], step);
            if (up) w[i] = got;
            else w[i + step] = got;
        }
}
// Bytes of four words as a 4 x 4 matrix, transposed.
__device__ __forceinline__ void transpose_bytes(uint32_t (&w)[4]) {
    const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[0], w[1], 0x7362);
    const uint32_t c = __byte_perm(w[2], w[3], 0x5140), d = __byte_perm(w[2], w[3], 0x7362);
    w[0] = __byte_perm(a, c, 0x5410);
    w[1] = __byte_perm(a, c, 0x7632);
    w[2] = __byte_perm(b, d, 0x5410);
    w[3] = __byte_perm(b, d, 0x7632);
}

template <bool F16>
__global__ void __launch_bounds__(kNT, 4) append_kernel(const RowPtr k, const RowPtr v, int n, int first_host,
                                                        const int32_t *first_dev, uint8_t *cache, int nb_cap,
                                                        uint32_t *flags) {
    __shared__ __align__(16) uint8_t tile[kQBlockTok * kPitch];   // V codes, [token][dimension]
    const int tid = threadIdx.x, c = tid & 3, tok = tid >> 2;
    const int g = blockIdx.y;
    const long long first = first_dev ? (long long)*first_dev : (long long)first_host;
    const long long cap = (long long)nb_cap * kQBlockTok;
    if (first_dev && blockIdx.x == 0 && g == 0 && tid == 0 && flags && (first < 0 || first + n > cap))
        atomicOr(flags, QSA_FLAG_NBLOCKS_CLAMPED);
    const long long b64 = (first >= 0 ? first / kQBlockTok : -((kQBlockTok - 1 - first) / kQBlockTok)) + blockIdx.x;
    if (b64 < 0 || b64 >= nb_cap) return;
    const int b = (int)b64;
    if ((long long)b * kQBlockTok >= first + n) return;
    const long long at = (long long)b * kQBlockTok - first;       // the row that the block's first token takes
    const long long i = at + tok;
    // the block's tokens t0 .. t1 - 1 are the call's
    const int t0 = at < 0 ? (int)min(-at, (long long)kQBlockTok) : 0;
    const int t1 = (int)min((long long)n - at, (long long)kQBlockTok);
    const bool in = tok >= t0 && tok < t1;
    uint8_t *rec = cache + qrec_offset(g, nb_cap, b);
    uint32_t xk[16], xv[16], packed[4];
    const uint8_t *krow = k.p + i * k.token_bytes + g * k.head_bytes;
    const uint8_t *vrow = v.p + i * v.token_bytes + g * v.head_bytes;
    if (in) {
        load_row(krow, c, xk);
        load_row(vrow, c, xv);
    } else {   // a token outside the range: zeros, so that its four threads agree
#pragma unroll
        for (int j = 0; j < 16; ++j) xk[j] = xv[j] = 0u;
    }
    const uint32_t kpair = quantise<F16>(xk, krow, c, packed);
    if (in) {
        uint2 *dst = reinterpret_cast<uint2 *>(rec + (c >> 1) * 1024 + tok * 16) + (c & 1);
        dst[0] = make_uint2(packed[0], packed[1]);
        dst[2 * 1024 / 8] = make_uint2(packed[2], packed[3]);
        if (c == 0) *reinterpret_cast<uint32_t *>(rec + kQOffKPair + tok * 4) = kpair;
    }
    const uint32_t vpair = quantise<F16>(xv, vrow, c, packed);
    if (in && c == 0) *reinterpret_cast<uint32_t *>(rec + kQOffVPair + tok * 4) = vpair;
    // unpacked to bytes
    uint2 *row = reinterpret_cast<uint2 *>(tile + tok * kPitch);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        row[c + 4 * j] = make_uint2(packed[2 * j] & 0x0F0F0F0Fu, packed[2 * j + 1] & 0x0F0F0F0Fu);
        row[8 + c + 4 * j] = make_uint2((packed[2 * j] >> 4) & 0x0F0F0F0Fu, (packed[2 * j + 1] >> 4) & 0x0F0F0F0Fu);
    }
    // V plane p, dimensions 4 d4 .. 4 d4 + 3: this thread takes tokens 16p + 4q .. + 3 (low nibbles) and those 32
    // further (high), then trades with its three neighbours for all 16 tokens of dimension 4 d4 + q
    const int p = tid >> 7, d4 = (tid & 127) >> 2, q = tid & 3;
    uint4 *dst = reinterpret_cast<uint4 *>(rec + kQOffV + p * 2048 + (4 * d4 + q) * 16);
    const bool whole = t1 - t0 == kQBlockTok;
    const uint4 old = whole ? make_uint4(0u, 0u, 0u, 0u) : __ldcg(dst);
    __syncthreads();
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(tile + (16 * p + 4 * q + j) * kPitch) + d4;
        w[j] = src[0] | (src[32 * kPitch / 4] << 4);
    }
    transpose_bytes(w);
    transpose_lanes(w, q);
    if (whole) {
        *dst = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
    // the other tokens' nibbles stay, also while another append writes them: in a word that holds both, what changes of
    // this call's own nibbles is flipped (nobody else writes those)
    uint32_t *word = reinterpret_cast<uint32_t *>(dst);
    const uint32_t was[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        uint32_t mine = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 16 * p + 4 * x + j;
            if (t >= t0 && t < t1) mine |= 0x0Fu << (8 * j);
            if (t + 32 >= t0 && t + 32 < t1) mine |= 0xF0u << (8 * j);
        }
        if (mine == ~0u) word[x] = w[x];
        else if (mine) atomicXor(word + x, (w[x] ^ was[x]) & mine);
    }
}

// 32 codes of a token (units c and c + 4 in lo, c + 8 and c + 12 in hi) to 16-bit values: scale * code + min
// rounded once.  The scale is rounded up, so the top level may pass the format's largest value, by half a step at
// most where a code stands for a finite value: then that value is what is read.
template <bool F16>
__device__ __forceinline__ void store_row(uint8_t *row, int c, const uint32_t (&lo)[4], const uint32_t (&hi)[4],
                                          uint32_t pair) {
    using Fmt = QFmt<F16>;
    const uint32_t scale2 = __byte_perm(pair, 0u, 0x1010), min2 = __byte_perm(pair, 0u, 0x3232);
    uint4 *r = reinterpret_cast<uint4 *>(row);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // a code's byte under the format's high byte is the base + code
            const uint32_t w = (i < 2 ? lo : hi)[2 * (i & 1) + (j >> 1)];
            const uint32_t code2 = Fmt::fma2(__byte_perm(w, Fmt::kCodeHigh, j & 1 ? 0x4342 : 0x4140), Fmt::kOne2, Fmt::kMinusBase2);
            o[j] = Fmt::min2(Fmt::fma2(scale2, code2, min2), Fmt::kMax2);   // min is finite: nothing passes below
        }
        r[c + 4 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <bool F16>
__global__ void __launch_bounds__(kNT) load_kernel(const uint8_t *cache, int nb_cap, int first, int n,
                                                   const RowPtrW k, const RowPtrW v) {
    __shared__ __align__(16) uint8_t tile[kQBlockTok * kPitch];
    const int tid = threadIdx.x, c = tid & 3, tok = tid >> 2;
    const int g = blockIdx.y, b = first / kQBlockTok + blockIdx.x;
    const uint8_t *rec = cache + qrec_offset(g, nb_cap, b);
    const long long i = (long long)b * kQBlockTok + tok - first;
    const bool in = i >= 0 && i < n;
    const int p = tid >> 7, d4 = (tid & 127) >> 2, q = tid & 3;
    const uint4 x = *reinterpret_cast<const uint4 *>(rec + kQOffV + p * 2048 + (4 * d4 + q) * 16);
    uint2 kx[2] = {};
    uint32_t kpair = 0u, vpair = 0u;
    if (in) {
        const uint2 *src = reinterpret_cast<const uint2 *>(rec + (c >> 1) * 1024 + tok * 16) + (c & 1);
        kx[0] = src[0];
        kx[1] = src[2 * 1024 / 8];
        kpair = *reinterpret_cast<const uint32_t *>(rec + kQOffKPair + tok * 4);
        vpair = *reinterpret_cast<const uint32_t *>(rec + kQOffVPair + tok * 4);
    }
    {   // V codes to shared memory, token-major (the writer's steps backwards)
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
        transpose_lanes(w, q);
        transpose_bytes(w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t *dst = reinterpret_cast<uint32_t *>(tile + (16 * p + 4 * q + j) * kPitch) + d4;
            dst[0] = w[j] & 0x0F0F0F0Fu;
            dst[32 * kPitch / 4] = (w[j] >> 4) & 0x0F0F0F0Fu;
        }
    }
    if (in) {
        const uint32_t w[4] = {kx[0].x, kx[0].y, kx[1].x, kx[1].y};
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            lo[j] = w[j] & 0x0F0F0F0Fu;
            hi[j] = (w[j] >> 4) & 0x0F0F0F0Fu;
        }
        store_row<F16>(k.p + i * k.token_bytes + g * k.head_bytes, c, lo, hi, kpair);
    }
    __syncthreads();
    if (in) {
        const uint2 *row = reinterpret_cast<const uint2 *>(tile + tok * kPitch);
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint2 a = row[c + 4 * j], e = row[8 + c + 4 * j];
            lo[2 * j] = a.x, lo[2 * j + 1] = a.y;
            hi[2 * j] = e.x, hi[2 * j + 1] = e.y;
        }
        store_row<F16>(v.p + i * v.token_bytes + g * v.head_bytes, c, lo, hi, vpair);
    }
}

}  // namespace

qsa_status launch_qcache_append(const QAppendArgs &a, cudaStream_t s) {
    const RowPtr k{static_cast<const uint8_t *>(a.k), 2 * a.k_token_stride, 2 * a.k_head_stride};
    const RowPtr v{static_cast<const uint8_t *>(a.v), 2 * a.v_token_stride, 2 * a.v_head_stride};
    // blocks the range touches; from a device position, at most one more than whole ones
    const int blocks = a.first_dev ? (a.n + 2 * kQBlockTok - 2) / kQBlockTok
                                   : (a.first + a.n - 1) / kQBlockTok - a.first / kQBlockTok + 1;
    const dim3 grid((unsigned)blocks, (unsigned)a.n_kv_heads);
    auto *kern = a.dt == QSA_F16 ? append_kernel<true> : append_kernel<false>;
    kern<<<grid, kNT, 0, s>>>(k, v, a.n, a.first, a.first_dev, static_cast<uint8_t *>(a.cache),
                              a.capacity / kQBlockTok, a.flags);
    return check_cuda(cudaGetLastError(), "append_kernel launch");
}

qsa_status launch_qcache_load(const QLoadArgs &a, cudaStream_t s) {
    const RowPtrW k{static_cast<uint8_t *>(a.k), 2 * a.k_token_stride, 2 * a.k_head_stride};
    const RowPtrW v{static_cast<uint8_t *>(a.v), 2 * a.v_token_stride, 2 * a.v_head_stride};
    const int blocks = (a.first + a.n - 1) / kQBlockTok - a.first / kQBlockTok + 1;
    const dim3 grid((unsigned)blocks, (unsigned)a.n_kv_heads);
    auto *kern = a.dt == QSA_F16 ? load_kernel<true> : load_kernel<false>;
    kern<<<grid, kNT, 0, s>>>(static_cast<const uint8_t *>(a.cache), a.capacity / kQBlockTok, a.first, a.n, k, v);
    return check_cuda(cudaGetLastError(), "load_kernel launch");
}

}  // namespace qsa
