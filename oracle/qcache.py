"""FP64 oracle of the 4-bit KV cache and the eviction (test infrastructure, CPU, numpy).

Rows, records, attention over them, block weights and the eviction plan as include/qsa.h
defines them; nothing here is shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

REC, KPAIR, VPAIR, VCODE = 8704, 4096, 4352, 4608
BLOCK, DIM = 64, 128
BF16, F16 = "bf16", "fp16"
_SIG = {BF16: (8, -133), F16: (11, -24)}   # significand bits, exponent of the least positive step


def bits_to_f64(bits: np.ndarray, fmt: str) -> np.ndarray:
    b = np.asarray(bits, dtype=np.uint16)
    if fmt == F16:
        return b.view(np.float16).astype(np.float64)
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bits(x: np.ndarray, fmt: str) -> np.ndarray:
    """Bits of values that the format holds exactly."""
    if fmt == F16:
        return np.asarray(x, dtype=np.float16).view(np.uint16)
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def round_up(x: np.ndarray, fmt: str) -> np.ndarray:
    """The least value of the format >= x, for x >= 0."""
    sig, least = _SIG[fmt]
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - sig, least))
    return np.ceil(x / step) * step


def quantise(x: np.ndarray, fmt: str):
    """codes [..., 128] uint8, scale [...], min [...] (float64) of rows x."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        lo, hi = x.min(-1), x.max(-1)
        wide = np.float64(np.finfo(np.float32).max)
        bad = ~(np.isfinite(x).all(-1)) | ~(hi - lo <= wide)
    lo, rng = np.where(bad, 0.0, lo) + 0.0, np.where(bad, 0.0, hi - lo)
    scale = round_up(rng / 15, fmt)
    with np.errstate(invalid="ignore", divide="ignore"):
        y = np.where((scale > 0)[..., None], (np.where(bad[..., None], 0.0, x) - lo[..., None]) / scale[..., None], 0.0)
    codes = np.clip(np.rint(y), 0, 15).astype(np.uint8)
    return codes, np.where(bad, np.nan, scale), np.where(bad, np.nan, lo)


def _nan_pair(fmt: str) -> int:
    return 0x7E007E00 if fmt == F16 else 0x7FC07FC0


def write_token(cache: np.ndarray, g: int, t: int, which: str, codes, scale, lo, fmt: str) -> None:
    """One token's row into cache [kv, blocks, REC] (uint8)."""
    rec, r = cache[g, t // BLOCK], t % BLOCK
    if np.isnan(scale):
        pair = _nan_pair(fmt)
    else:
        pair = int(f64_to_bits(scale, fmt)) | (int(f64_to_bits(lo, fmt)) << 16)
    at = (KPAIR if which == "k" else VPAIR) + 4 * r
    rec[at:at + 4] = np.frombuffer(np.uint32(pair).tobytes(), dtype=np.uint8)
    for d in range(DIM):
        if which == "k":
            off, high = ((d % 64) // 16) * 1024 + r * 16 + d % 16, d >= 64
        else:
            off, high = VCODE + ((r % 32) // 16) * 2048 + d * 16 + r % 16, r >= 32
        old = int(rec[off])
        rec[off] = (old & 0x0F) | (int(codes[d]) << 4) if high else (old & 0xF0) | int(codes[d])


def append(cache: np.ndarray, k: np.ndarray, v: np.ndarray, first: int, fmt: str) -> None:
    """k, v [n, kv, 128] (16-bit values as float64) into positions first .."""
    cap = cache.shape[1] * BLOCK
    for which, x in (("k", k), ("v", v)):
        codes, scale, lo = quantise(x, fmt)
        for i in range(x.shape[0]):
            if 0 <= first + i < cap:
                for g in range(x.shape[1]):
                    write_token(cache, g, first + i, which, codes[i, g], scale[i, g], lo[i, g], fmt)


def read_block(rec: np.ndarray, fmt: str):
    """(K codes [64,128], V codes [64,128], pairs [2,64,2] of (scale, min)) of a record, float64."""
    kp = rec[:KPAIR].reshape(4, BLOCK, 16)
    kc = np.concatenate([(kp & 15).transpose(1, 0, 2).reshape(BLOCK, 64), (kp >> 4).transpose(1, 0, 2).reshape(BLOCK, 64)],
                        axis=1)
    vp = rec[VCODE:].reshape(2, DIM, 16)
    vc = np.concatenate([(vp & 15).transpose(0, 2, 1).reshape(32, DIM), (vp >> 4).transpose(0, 2, 1).reshape(32, DIM)])
    pairs = bits_to_f64(np.ascontiguousarray(rec[KPAIR:VCODE]).view(np.uint16), fmt).reshape(2, BLOCK, 2)
    return kc.astype(np.float64), vc.astype(np.float64), pairs


def rows(cache: np.ndarray, first: int, n: int, fmt: str):
    """K and V values [n, kv, 128] of positions first .., float64, not rounded."""
    kv = cache.shape[0]
    k, v = np.empty((n, kv, DIM)), np.empty((n, kv, DIM))
    for g in range(kv):
        for b in range(first // BLOCK, (first + n - 1) // BLOCK + 1 if n else 0):
            kc, vc, pairs = read_block(cache[g, b], fmt)
            for r in range(BLOCK):
                i = b * BLOCK + r - first
                if 0 <= i < n:
                    k[i, g] = pairs[0, r, 0] * kc[r] + pairs[0, r, 1]
                    v[i, g] = pairs[1, r, 0] * vc[r] + pairs[1, r, 1]
    return k, v


def attention(q: np.ndarray, cache: np.ndarray, ids: np.ndarray, n_tokens: np.ndarray, scale: float, fmt: str):
    """out [nq, H, 128], lse [nq, H], weights [nq, kv, k], and what bounds their errors:
    dict(mass [nq, H, 128] = sum w |V - min|, least [nq, H] = sum w |min|, top [nq, H] largest weight, vstep [nq, kv] largest V
    scale, tokens [nq], logit [nq, H] = largest sum |q| (|K - min| + |min|) times scale)."""
    nq, heads, _ = q.shape
    kv, cap = cache.shape[0], cache.shape[1] * BLOCK
    group, k = heads // kv, ids.shape[1]
    out, lse = np.zeros((nq, heads, DIM)), np.full((nq, heads), -np.inf)
    weights = np.zeros((nq, kv, k))
    info = dict(mass=np.zeros((nq, heads, DIM)), least=np.zeros((nq, heads)), top=np.zeros((nq, heads)), vstep=np.zeros((nq, kv)),
                tokens=np.zeros(nq), logit=np.zeros((nq, heads)))
    for i in range(nq):
        nt = int(min(max(int(n_tokens[i]), 0), cap))
        nb = (nt + BLOCK - 1) // BLOCK
        slots, seen = [], set()
        for j in range(k):
            b = int(ids[i, j])
            if 0 <= b < nb and b not in seen:
                seen.add(b)
                slots.append(j)
        if not slots:
            continue
        for g in range(kv):
            ks, ka, vs, vd, vm, at, step = [], [], [], [], [], [], 0.0
            for j in slots:
                b = int(ids[i, j])
                m = min(BLOCK, nt - b * BLOCK)
                kc, vc, pr = read_block(cache[g, b], fmt)
                ks.append((pr[0, :, :1] * kc + pr[0, :, 1:])[:m])
                ka.append((pr[0, :, :1] * kc + np.abs(pr[0, :, 1:]))[:m])
                vs.append((pr[1, :, :1] * vc + pr[1, :, 1:])[:m])
                vd.append((pr[1, :, :1] * vc)[:m])
                vm.append(np.abs(pr[1, :m, 1]))
                at += [j] * m
                step = max(step, float(pr[1, :m, 0].max()))
            K, A, V, Vd, Vm = (np.concatenate(x) for x in (ks, ka, vs, vd, vm))
            at = np.array(at)
            for h in range(g * group, (g + 1) * group):
                s = scale * (K @ q[i, h])
                m = s.max()
                p = np.exp(s - m)
                tot = p.sum()
                w = p / tot
                out[i, h], lse[i, h] = w @ V, m + np.log(tot)
                np.add.at(weights[i, g], at, w)
                info["mass"][i, h], info["least"][i, h], info["top"][i, h] = w @ Vd, w @ Vm, w.max()
                info["logit"][i, h] = scale * (A @ np.abs(q[i, h])).max()
            info["vstep"][i, g] = step
        info["tokens"][i] = len(at)
    return out, lse, weights, info


def weights_add(weights: np.ndarray, ids: np.ndarray, decay: float, prev, n: int) -> np.ndarray:
    acc = np.zeros(n) if prev is None else decay * prev.astype(np.float64)
    for i in range(ids.shape[0]):
        for j in range(ids.shape[1]):
            if 0 <= ids[i, j] < n:
                acc[ids[i, j]] += weights[i, :, j].astype(np.float64).sum()
    return acc


def evict_plan(weights: np.ndarray, n_tokens: int, n_keep: int, n_first: int, n_last: int):
    """(kept ids ascending with -1 behind, tokens left) of one row of weights."""
    nb = (n_tokens + BLOCK - 1) // BLOCK
    if nb <= n_keep:
        return np.array(list(range(nb)) + [-1] * (n_keep - nb), dtype=np.int32), n_tokens
    must = set(range(n_first)) | set(range(nb - n_last, nb))
    rest = sorted((b for b in range(nb) if b not in must),
                  key=lambda b: (0, -float(weights[b]), b) if not np.isnan(weights[b]) else (1, 0.0, b))
    kept = sorted(must | set(rest[:n_keep - len(must)]))
    return np.array(kept, dtype=np.int32), n_tokens - BLOCK * (nb - n_keep)
