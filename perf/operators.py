"""Cases of the 4-bit KV cache and its eviction: what each operator computes, in plain torch
operations and through the library, on inputs of real sizes.

Four operators:

* ``append``     K and V rows of new tokens quantised into the 4-bit block cache, and read back;
* ``attend``     selection attention over the 4-bit cache (output, log-sum-exp, and each selected
                 block's share of the attention);
* ``accumulate`` those shares added up per block, with a decay;
* ``evict``      the blocks to keep by accumulated share, and their records moved together.

The cache is ``[n_kv_heads][blocks][8704]`` bytes, one record per 64-token block: K codes (4 planes of
[64 tokens][16 bytes]; byte j of plane c holds dimension 16c + j in its low nibble and 64 + 16c + j in
its high one), 64 K pairs (scale, minimum) in 16 bits, 64 V pairs, V codes (2 planes of [128 dimensions]
[16 bytes]; byte j of plane c holds token 16c + j low and 32 + 16c + j high).  A value is
scale x code + minimum; scale is the least 16-bit number at or above (max - min) / 15 of the token's
row, and the code is (x - min) / scale rounded half to even.
"""
import math

import torch

own = False

D = 128          # head dimension
BT = 64          # tokens of a block
REC = 8704       # bytes of a block's record
KP, VP, VC = 4096, 4352, 4608   # offsets of the K pairs, the V pairs and the V codes in a record

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's write: one token's K and V, slices of a fused projection row, behind 258,000 tokens
        {"name": "append 1 token", "op": "append", "n": 1, "first": 257_999, "kv": 4, "dt": "bf16", "fused": True},
        # a ragged prompt chunk whose first and last blocks are partial
        {"name": "append 255 tokens", "op": "append", "n": 255, "first": 1017, "kv": 4, "dt": "fp16", "fused": True},
        # a whole prompt
        {"name": "append 131072 tokens", "op": "append", "n": 131_072, "first": 0, "kv": 4, "dt": "bf16", "fused": False},
        # the decode step of one sequence at 258,000 tokens: latency
        {"name": "attend 1 query", "op": "attend", "nq": 1, "kv": 4, "group": 16, "tokens": 258_000, "k": 32,
         "dt": "bf16", "weights": False, "ragged": False},
        # a decode window of three queries with the largest selection
        {"name": "attend 3 queries k64", "op": "attend", "nq": 3, "kv": 4, "group": 16, "tokens": 258_000, "k": 64,
         "dt": "fp16", "weights": True, "ragged": False},
        # eight KV heads of eight heads, ragged contexts, an odd selection
        {"name": "attend 61 ragged", "op": "attend", "nq": 61, "kv": 8, "group": 8, "tokens": 131_072, "k": 17,
         "dt": "fp16", "weights": True, "ragged": True},
        # the prompt chunk over the deep context
        {"name": "attend 256 deep", "op": "attend", "nq": 256, "kv": 4, "group": 16, "tokens": 520_000, "k": 32,
         "dt": "bf16", "weights": True, "ragged": False},
        # the shares of a decode window
        {"name": "accumulate 3 queries", "op": "accumulate", "nq": 3, "kv": 4, "k": 32, "blocks": 4032, "decay": 0.98},
        # the shares of a prompt chunk over the deep context
        {"name": "accumulate 256 queries", "op": "accumulate", "nq": 256, "kv": 4, "k": 32, "blocks": 8125, "decay": 0.9},
        # a short context of one KV head halved
        {"name": "evict to 128 blocks", "op": "evict", "blocks": 257, "tail": 5, "keep": 128, "first": 1, "last": 8,
         "kv": 1, "wide": False},
        # the deep context halved, 4-bit records and indexer keys
        {"name": "evict deep to 4096", "op": "evict", "blocks": 8125, "tail": 64, "keep": 4096, "first": 4, "last": 64,
         "kv": 4, "wide": False},
        # a 16-bit cache (K rows and V blocks) and its indexer keys, an odd number kept
        {"name": "evict 16-bit to 1111", "op": "evict", "blocks": 2048, "tail": 64, "keep": 1111, "first": 4, "last": 32,
         "kv": 4, "wide": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "accumulate", "evict"])
    if op == "append":
        kv = rng.choice([1, 2, 4, 8])
        n = _log(rng, 1, 400_000 // kv)
        return {"op": op, "n": n, "first": rng.randrange(0, 4096), "kv": kv, "dt": rng.choice(["bf16", "fp16"]),
                "fused": rng.random() < 0.5 and n <= 8192}
    if op == "attend":
        kv = rng.choice([1, 2, 4, 8])
        k = _log(rng, 1, 64)
        nq = _log(rng, 1, min(256, 32_768 // (kv * k)))
        return {"op": op, "nq": nq, "kv": kv, "group": rng.choice([1, 4, 7, 8, 16]), "tokens": _log(rng, 65, 520_000), "k": k,
                "dt": rng.choice(["bf16", "fp16"]), "weights": rng.random() < 0.5, "ragged": rng.random() < 0.5}
    if op == "accumulate":
        return {"op": op, "nq": _log(rng, 1, 1024), "kv": rng.choice([1, 2, 4, 8]), "k": _log(rng, 1, 64),
                "blocks": _log(rng, 64, 16_384), "decay": round(rng.uniform(0.5, 1.0), 3)}
    blocks = _log(rng, 64, 8192)
    keep = rng.randrange(blocks // 4, blocks)
    return {"op": op, "blocks": blocks, "tail": rng.randrange(1, 65), "keep": keep, "first": rng.randrange(0, 5),
            "last": rng.randrange(1, max(2, keep // 8)), "kv": rng.choice([1, 2, 4]), "wide": blocks <= 2048 and rng.random() < 0.4}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _cache(g, kv, blocks, dt):
    """A filled 4-bit cache: codes of about normal rows, scales and minima to go with them."""
    c = torch.empty(kv, blocks, REC, dtype=torch.uint8, device="cuda")
    for at, n in ((0, KP), (VC, REC - VC)):
        for h in range(kv):
            lo = torch.randn(blocks, n, device="cuda", generator=g).mul_(2.9).add_(7.5).round_().clamp_(0, 15)
            hi = torch.randn(blocks, n, device="cuda", generator=g).mul_(2.9).add_(7.5).round_().clamp_(0, 15)
            c[h, :, at:at + n] = (lo + 16 * hi).to(torch.uint8)
    pairs = torch.empty(kv, blocks, 2 * BT, 2, dtype=dt, device="cuda")
    scale = torch.rand(kv, blocks, 2 * BT, device="cuda", generator=g).mul_(0.16).add_(0.27)
    pairs[..., 0] = scale
    pairs[..., 1] = -scale * (torch.rand(kv, blocks, 2 * BT, device="cuda", generator=g).mul_(2.0).add_(6.5))
    c[:, :, KP:VC] = pairs.view(kv, blocks, 4 * BT).view(torch.uint8)
    return c


def _ids(g, n_tokens, nb_most, k, pads):
    """Distinct ascending block ids per query (int32, -1 behind them), the last block among most of them."""
    nq = n_tokens.numel()
    nb = (n_tokens.long() + BT - 1) // BT
    rank = torch.rand(nq, nb_most, device="cuda", generator=g)
    at = torch.arange(nb_most, device="cuda")
    rank[at[None] == (nb - 1)[:, None]] = 1.5
    rank[at[None] >= nb[:, None]] = -1.0
    top, ids = rank.topk(min(k, nb_most), dim=1)
    ids = torch.where(top >= 0, ids, nb_most)
    if pads:   # some queries select fewer blocks, every eleventh one none
        few = torch.randint(0, k + 1, (nq, 1), device="cuda", generator=g)
        few[torch.arange(nq, device="cuda") % 11 == 10] = 0
        few[torch.arange(nq, device="cuda") % 3 == 0] = k
        ids = torch.where(torch.arange(ids.shape[1], device="cuda")[None] < few, ids, nb_most)
    ids = ids.sort(dim=1).values
    out = torch.full((nq, k), -1, dtype=torch.int32, device="cuda")
    out[:, :ids.shape[1]] = torch.where(ids < nb_most, ids, -1).int()
    return out


def _rows(case, seed):
    """K and V rows [n][kv][128] of new tokens: normal rows with an offset and a few large dimensions."""
    g = _gen(seed)
    n, kv, dt = case["n"], case["kv"], _DT[case["dt"]]
    if case["fused"]:   # slices of a projection's rows: 16 query heads per KV head, then K, then V
        row = torch.randn(n, 18 * kv, D, device="cuda", generator=g).to(dt)
        k, v = row[:, 16 * kv:17 * kv], row[:, 17 * kv:]
    else:
        k = torch.randn(n, kv, D, device="cuda", generator=g).to(dt)
        v = torch.randn(n, kv, D, device="cuda", generator=g).to(dt)
    k[..., ::37] *= 4
    v += 0.25
    return k, v


def prepare(case, seed):
    op = case["op"]
    s = {"op": op}
    if op == "append":
        s["k"], s["v"] = _rows(case, seed)
        blocks = (case["first"] + case["n"] + BT - 1) // BT
        s["first"] = case["first"]
        s["cache"] = torch.zeros(case["kv"], blocks, REC, dtype=torch.uint8, device="cuda")
        s["k_out"], s["v_out"] = (torch.empty(case["n"], case["kv"], D, dtype=_DT[case["dt"]], device="cuda") for _ in "kv")
        return s
    g = _gen(seed)
    if op == "attend":
        nq, kv, k, dt, tokens = case["nq"], case["kv"], case["k"], _DT[case["dt"]], case["tokens"]
        blocks = (tokens + BT - 1) // BT
        s["cache"] = _cache(g, kv, blocks, dt)
        n = torch.full((nq,), tokens, dtype=torch.int32, device="cuda")
        if case["ragged"]:
            n = torch.randint(1, tokens + 1, (nq,), device="cuda", generator=g, dtype=torch.int32)
        s["n_tokens"] = n
        s["ids"] = _ids(g, n, blocks, k, case["ragged"])
        s["q"] = torch.randn(nq, kv * case["group"], D, device="cuda", generator=g).mul_(1.25).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(nq, kv * case["group"], device="cuda")
        s["weights"] = torch.empty(nq, kv, k, device="cuda") if case["weights"] else None
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    elif op == "accumulate":
        nq, kv, k, blocks = case["nq"], case["kv"], case["k"], case["blocks"]
        n = torch.full((nq,), blocks * BT, dtype=torch.int32, device="cuda")
        s["ids"] = _ids(g, n, blocks, k, False)
        w = torch.rand(nq, kv, k, device="cuda", generator=g).pow_(4)
        s["weights"] = w * (16 / w.sum(-1, keepdim=True))   # 16 heads' probabilities over the selection
        s["prev"] = torch.rand(blocks, device="cuda", generator=g).pow_(6).mul_(100)
        s["acc"] = torch.empty(blocks, device="cuda")
        s["decay"] = case["decay"]
    else:
        kv, blocks, keep = case["kv"], case["blocks"], case["keep"]
        w = torch.rand(blocks, device="cuda", generator=g).pow_(6).mul_(100)
        s["acc"] = torch.where(torch.rand(blocks, device="cuda", generator=g) < 0.2, 0.0, w)   # never selected: ties at 0
        s["n_tokens"] = torch.tensor([(blocks - 1) * BT + case["tail"]], dtype=torch.int32, device="cuda")
        kblk = torch.randn(blocks, D, device="cuda", generator=g).bfloat16()
        if case["wide"]:
            src = [torch.randn(kv, blocks, BT * D, device="cuda", generator=g).bfloat16() for _ in "kv"]
        else:
            src = [_cache(g, kv, blocks, torch.bfloat16)]
        s["src"] = src + [kblk, s["acc"]]
        s["dst"] = [torch.zeros(x.shape[0], keep, x.shape[2], dtype=x.dtype, device="cuda") for x in src]
        s["dst"] += [torch.zeros(keep, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(keep, device="cuda")]
        s["keep"] = torch.empty(1, keep, dtype=torch.int32, device="cuda")
        s["new_tokens"] = torch.empty(1, dtype=torch.int32, device="cuda")
        s["first"], s["last"] = case["first"], case["last"]
    return s


# ------------------------------------------------------------------ one pass

def _round_up(x, dt):
    """The least value of type dt at or above x >= 0 (float64)."""
    y = x.to(dt)
    return torch.where(y.double() < x, (y.view(torch.int16) + 1).view(dt), y)


def _quantised(x):
    """x rounded to its row's 16 levels, in x's type (64 bits inside: codes lie next to borders)."""
    r = x.double()
    lo = r.amin(-1, keepdim=True)
    scale = _round_up((r.amax(-1, keepdim=True) - lo) / 15, x.dtype).double()
    code = ((r - lo) / torch.where(scale > 0, scale, 1.0)).round_().clamp_(0, 15)
    return (code * scale + lo).to(x.dtype)


def _planes(codes):
    """[..., planes, rows, 16] packed bytes -> [..., 2 planes, rows, 16] codes, the low nibbles first."""
    return torch.cat((codes & 15, codes >> 4), dim=-3)


def _attend(q, cache, ids, n_tokens, want_weights):
    nq, heads, _ = q.shape
    kv = cache.shape[0]
    k = ids.shape[1]
    rec = cache[:, ids.long().clamp(min=0)]                                        # [kv, nq, k, REC]
    pairs = rec[..., KP:VC].contiguous().view(q.dtype).view(kv, nq, k, 2, BT, 2).float()
    kc = _planes(rec[..., :KP].unflatten(-1, (4, BT, 16)))                         # [.., 8, 64, 16]
    kc = kc.transpose(-3, -2).reshape(kv, nq, k, BT, D).float()
    keys = (kc * pairs[..., 0, :, :1] + pairs[..., 0, :, 1:]).view(kv, nq, k * BT, D)
    vc = _planes(rec[..., VC:].unflatten(-1, (2, D, 16)))                          # [.., 4, 128, 16]
    vc = vc.transpose(-2, -1).reshape(kv, nq, k, BT, D).float()
    vals = (vc * pairs[..., 1, :, :1] + pairs[..., 1, :, 1:]).view(kv, nq, k * BT, D)
    qs = q.float().view(nq, kv, heads // kv, D).transpose(0, 1)                    # [kv, nq, group, D]
    s = (qs @ keys.transpose(-1, -2)) * D ** -0.5
    t = ids.long()[:, :, None] * BT + torch.arange(BT, device=q.device)
    seen = ((ids >= 0)[:, :, None] & (t < n_tokens[:, None, None])).view(1, nq, 1, k * BT)
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    r = {"out": (p @ vals).transpose(0, 1).reshape(nq, heads, D).to(q.dtype),
         "lse": (m + torch.log(total)).transpose(0, 1).reshape(nq, heads)}
    if want_weights:
        r["weights"] = p.view(kv, nq, heads // kv, k, BT).sum((2, 4)).transpose(0, 1)
    return r


def _evicted(s):
    acc, keep = s["acc"], s["keep"].shape[1]
    n = s["n_tokens"].long()
    nb = (n + BT - 1) // BT
    at = torch.arange(acc.numel(), device="cuda")
    key = torch.where((at < s["first"]) | (at >= nb - s["last"]), math.inf, acc)
    key = torch.where(at < nb, key, -math.inf)
    ids = key.sort(descending=True, stable=True).indices[:keep].sort().values
    kept = torch.where(ids < nb, ids, -1)
    moved = [x.index_select(x.dim() - 2 if x.dim() > 1 else 0, ids) for x in s["src"]]
    return {"keep": kept[None].int(), "new_tokens": (n - BT * (nb - torch.clamp(nb, max=keep))).int(), "moved": moved}


def run(s):
    op = s["op"]
    if own:
        from sparse_attention_kv_gb300 import qsa
        if op == "append":
            qsa.qcache_append(s["k"], s["v"], s["cache"], s["first"])
            qsa.qcache_load(s["cache"], s["k_out"], s["v_out"], s["first"])
            return {"k": s["k_out"], "v": s["v_out"]}
        if op == "attend":
            qsa.select_attention_qcache(s["q"], s["cache"], s["ids"], s["n_tokens"], s["out"], s["lse"], s["weights"], ws=s["ws"])
            r = {"out": s["out"], "lse": s["lse"]}
            if s["weights"] is not None:
                r["weights"] = s["weights"]
            return r
        if op == "accumulate":
            qsa.block_weights_add(s["weights"], s["ids"], s["acc"], prev=s["prev"], decay=s["decay"])
            return s["acc"]
        qsa.evict_plan(s["acc"][None], s["n_tokens"], s["keep"], s["new_tokens"], n_first=s["first"], n_last=s["last"])
        qsa.gather_blocks(list(zip(s["src"], s["dst"])), s["keep"][0])
        return {"keep": s["keep"], "new_tokens": s["new_tokens"], "moved": s["dst"]}
    if op == "append":
        return {"k": _quantised(s["k"]), "v": _quantised(s["v"])}
    if op == "attend":
        return _attend(s["q"], s["cache"], s["ids"], s["n_tokens"], s["weights"] is not None)
    if op == "accumulate":
        add = torch.zeros_like(s["prev"], dtype=torch.float64)   # long sums of unlike terms
        add.index_add_(0, s["ids"].long().clamp(min=0).reshape(-1),
                       torch.where(s["ids"] >= 0, s["weights"].double().sum(1), 0.0).reshape(-1))
        return (s["prev"].double() * s["decay"] + add).float()
    return _evicted(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "append":   # rows in, codes and pairs written, read again, rows out
        rows = case["n"] * case["kv"] * 2
        return {"bytes": rows * (256 + 68 + 68 + 256), "flops": rows * D * 6}
    if op == "attend":
        nq, kv, k, heads = case["nq"], case["kv"], case["k"], case["kv"] * case["group"]
        nb = (case["tokens"] + BT - 1) // BT
        mean_k = min(k, nb) * (0.6 if case["ragged"] else 1.0)
        distinct = nb * (1 - (1 - mean_k / nb) ** nq)          # blocks that some query selects
        b = distinct * kv * REC + nq * heads * (2 * 2 * D + 4) + nq * (4 * k + 4) + (4 * nq * kv * k if case["weights"] else 0)
        return {"bytes": b, "flops": 4 * nq * heads * mean_k * BT * D}
    if op == "accumulate":
        e = case["nq"] * case["k"]
        return {"bytes": e * 4 + e * case["kv"] * 4 + case["blocks"] * 8, "flops": e * case["kv"] + 2 * case["blocks"]}
    row = (case["kv"] * (4 * BT * D if case["wide"] else REC) + 2 * D + 4) * case["keep"]
    return {"bytes": 2 * row + case["blocks"] * 4 + case["keep"] * 4, "flops": case["blocks"]}


# ------------------------------------------------------------------ the definition in 64 bits

_SIG = {"bf16": (8, -133), "fp16": (11, -24)}   # significand bits, exponent of the least step


def _levels(x, dt):
    """Rows x (float64) at their 16 levels: scale by the mantissa rounded up, codes by distance."""
    bits, least = _SIG[dt]
    lo = x.min(-1, keepdim=True).values
    want = (x.max(-1, keepdim=True).values - lo) / 15
    step = torch.exp2(torch.clamp(torch.frexp(want).exponent - bits, min=least).double())
    scale = torch.ceil(want / step) * step
    y = torch.where(scale > 0, (x - lo) / scale, 0.0)
    f = torch.floor(y)
    code = f + ((y - f > 0.5) | ((y - f == 0.5) & (f % 2 == 1)))
    return scale * code.clamp(max=15) + lo


def _exact_attend(case, s):
    q, cache, ids, n_tokens = s["q"].double(), s["cache"], s["ids"].cpu(), s["n_tokens"].cpu()
    nq, heads, _ = q.shape
    kv = cache.shape[0]
    group = heads // kv
    t, d = torch.meshgrid(torch.arange(BT, device="cuda"), torch.arange(D, device="cuda"), indexing="ij")
    k_at, k_shift = ((d % 64) // 16) * 1024 + t * 16 + d % 16, (d // 64) * 4
    v_at, v_shift = VC + ((t % 32) // 16) * 2048 + d * 16 + t % 16, (t // 32) * 4
    out = torch.zeros(nq, heads, D, dtype=torch.float64, device="cuda")
    lse = torch.full((nq, heads), -math.inf, dtype=torch.float64, device="cuda")
    w = torch.zeros(nq, kv, ids.shape[1], dtype=torch.float64, device="cuda")
    for i in range(nq):
        slots = [j for j in range(ids.shape[1]) if ids[i, j] >= 0]
        if not slots:
            continue
        b = ids[i, slots].long().cuda()
        seen = (b[:, None] * BT + torch.arange(BT, device="cuda") < int(n_tokens[i])).reshape(-1)
        rec = cache[:, b]                                                           # [kv, m, REC]
        pairs = rec[..., KP:VC].contiguous().view(_DT[case["dt"]]).view(kv, len(slots), 2, BT, 2).double()
        key = ((rec[..., k_at] >> k_shift) & 15).double() * pairs[:, :, 0, :, :1] + pairs[:, :, 0, :, 1:]
        val = ((rec[..., v_at] >> v_shift) & 15).double() * pairs[:, :, 1, :, :1] + pairs[:, :, 1, :, 1:]
        z = torch.einsum("ghd,gtd->ght", q[i].view(kv, group, D), key.reshape(kv, -1, D)) / math.sqrt(D)
        z[:, :, ~seen] = -math.inf
        lse[i] = torch.logsumexp(z, -1).reshape(-1)
        p = torch.softmax(z, -1)
        out[i] = torch.einsum("ght,gtd->ghd", p, val.reshape(kv, -1, D)).reshape(heads, D)
        w[i][:, slots] = p.view(kv, group, len(slots), BT).sum((1, 3))
    r = {"out": out, "lse": lse}
    if case["weights"]:
        r["weights"] = w
    return r


def exact(case, seed):
    op = case["op"]
    if op == "append":
        return {n: torch.cat([_levels(x.double(), case["dt"]) for x in rows.split(16_384)])
                for n, rows in zip("kv", _rows(case, seed))}
    if op == "evict":   # whole numbers and moved bytes only
        return None
    s = prepare(case, seed)
    if op == "attend":
        return _exact_attend(case, s)
    ids, w = s["ids"].cpu().reshape(-1).tolist(), s["weights"].cpu().double().sum(1).reshape(-1).tolist()
    acc = [x * case["decay"] for x in s["prev"].cpu().double().tolist()]
    for b, x in zip(ids, w):
        if b >= 0:
            acc[b] += x
    return torch.tensor(acc, dtype=torch.float64)
