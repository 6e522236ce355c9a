"""Cases of the paged 16-bit KV cache: the attention of whole prompts, the attention of drafted token
trees over the pages, and the pages themselves, in plain torch operations and through the library.

Three operators:

* ``prompt``  causal attention of packed sequences: query i of a sequence with lq queries and lk keys
              sees its first lk - lq + i + 1 keys (a whole prompt has lk = lq, a chunk behind earlier
              tokens lk > lq);
* ``tree``    attention of drafted tokens: each sees the sequence's context, which lies in pages, and
              its own ancestors in a tree of drafts (one node: an ordinary decode step);
* ``pages``   the pages of a pool: rows appended behind reserved pages (``commit``), sequences dropped
              and forked with their shared last page copied before it is written (``fork``), live pages
              moved together (``compact``).

A page is a block of 64 tokens: K rows ``kcache[g][64 p ..][128]``, V ``vcache_t[g][p][128][64]`` with
the dimension before the token.  ``table[s]`` lists the pages of sequence s in order (-1 behind them),
``refs[p]`` counts the tables that hold page p.
"""
import math

import torch

own = False

D = 128          # head dimension
BT = 64          # tokens of a page

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few short requests of a serving batch, one of them a single token: latency
        {"name": "prompt 5 short", "op": "prompt", "lens": "1 17 64 130 300", "extra": "0 0 0 0 0", "kv": 4, "group": 16,
         "dt": "bf16", "fused": True},
        # a ragged batch with seven heads per KV head; two of its prompts continue earlier tokens
        {"name": "prompt 6 ragged", "op": "prompt", "lens": "1021 2047 333 1 1500 777", "extra": "0 0 517 2000 0 63", "kv": 2,
         "group": 7, "dt": "fp16", "fused": False},
        # a prompt chunk of 256 tokens at the end of a 131,072-token context
        {"name": "prompt chunk 256 of 131072", "op": "prompt", "lens": "256", "extra": "130816", "kv": 4, "group": 16,
         "dt": "bf16", "fused": False},
        # a whole long prompt
        {"name": "prompt 16384", "op": "prompt", "lens": "16384", "extra": "0", "kv": 4, "group": 16, "dt": "bf16",
         "fused": True},
        # the decode step of one sequence at 258,000 tokens
        {"name": "tree 1 node 258000", "op": "tree", "seqs": 1, "nodes": 1, "tokens": 258_000, "ragged": False, "kv": 4,
         "group": 16, "dt": "bf16"},
        # five sequences with small trees over short ragged contexts: latency
        {"name": "tree 5 short", "op": "tree", "seqs": 5, "nodes": 7, "tokens": 900, "ragged": True, "kv": 2, "group": 7,
         "dt": "fp16"},
        # a serving batch: 64 sequences, up to 8 drafts each, ragged contexts, eight KV heads of eight heads
        {"name": "tree batch of 64", "op": "tree", "seqs": 64, "nodes": 8, "tokens": 16_000, "ragged": True, "kv": 8,
         "group": 8, "dt": "bf16"},
        # the largest tree over a long context
        {"name": "tree 64 nodes 131072", "op": "tree", "seqs": 1, "nodes": 64, "tokens": 131_072, "ragged": False, "kv": 4,
         "group": 16, "dt": "bf16"},
        # the accepted drafts of eight sequences enter their pages
        {"name": "commit 8 trees", "op": "commit", "seqs": 8, "nodes": 16, "tokens": 8000, "kv": 4, "dt": "bf16", "pages": 2048},
        # a whole prompt enters its pages
        {"name": "commit 131072 tokens", "op": "commit", "seqs": 1, "nodes": 131_072, "tokens": 50, "kv": 4, "dt": "fp16",
         "pages": 4096},
        # a step of parallel sampling: eight sequences forked seven times each, the last page of each copied
        {"name": "fork 8 to 64", "op": "fork", "parents": 8, "ways": 7, "tokens": 6000, "kv": 4, "pages": 2048},
        # a pool with holes moved together
        {"name": "compact 4096 pages", "op": "compact", "seqs": 32, "kv": 4, "pages": 4096, "live": 0.55},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "commit", "fork", "compact"])
    dt = rng.choice(["bf16", "fp16"])
    if op == "prompt":
        seqs = _log(rng, 1, 12)
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8, 16])
        lens, extra, pairs = [], [], 1 << 33
        for _ in range(seqs):   # a drawn batch has at most the listed prompt's (query, key, head) triples
            most = int(math.sqrt(pairs / (seqs * kv * group)))
            n = _log(rng, 1, min(12_000, most))
            more = rng.choice([0, 0, _log(rng, 1, max(1, min(60_000, pairs // (2 * seqs * kv * group * n))))])
            lens.append(n)
            extra.append(-rng.randrange(0, n + 1) if rng.random() < 0.08 else more)   # fewer keys than queries: empty rows
        return {"op": op, "lens": " ".join(map(str, lens)), "extra": " ".join(map(str, extra)), "kv": kv, "group": group,
                "dt": dt, "fused": rng.random() < 0.5}
    if op == "tree":
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8, 16])
        seqs, nodes = _log(rng, 1, 48), _log(rng, 1, 64)
        most = (1 << 29) // (seqs * nodes * kv * group)
        return {"op": op, "seqs": seqs, "nodes": nodes, "tokens": _log(rng, 1, max(1, min(most, 1_000_000 // (seqs * kv)))),
                "ragged": rng.random() < 0.6, "kv": kv, "group": group, "dt": dt}
    kv = rng.choice([1, 2, 4])
    if op == "commit":
        seqs = _log(rng, 1, 64)
        nodes, tokens = _log(rng, 1, 100_000 // (kv * seqs)), rng.randrange(0, 4000)
        return {"op": op, "seqs": seqs, "nodes": nodes, "tokens": tokens, "kv": kv, "dt": dt,
                "pages": seqs * ((tokens + nodes) // BT + 2) + rng.randrange(0, 200)}
    if op == "fork":
        parents, ways, tokens = _log(rng, 1, 24), _log(rng, 1, 8), _log(rng, 1, 9000)
        return {"op": op, "parents": parents, "ways": ways, "tokens": tokens, "kv": kv,
                "pages": parents * (tokens // BT + 3) + 4 * parents * ways + rng.randrange(0, 300)}
    return {"op": op, "seqs": _log(rng, 1, 100), "kv": kv, "pages": _log(rng, 100, 4096), "live": round(rng.uniform(0.1, 0.95), 2)}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _cpu_gen(seed):
    return torch.Generator().manual_seed(int(seed))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _normal(g, *shape, dt, mean=0.0):
    return torch.randn(*shape, device="cuda", generator=g).add_(mean).to(dt)


def _lens(case):
    lq = [int(x) for x in case["lens"].split()]
    return lq, [n + int(x) for n, x in zip(lq, case["extra"].split())]


def _pool(g, kv, pages, dt):
    """A pool of filled pages: K rows and V blocks."""
    k = torch.empty(kv, pages * BT, D, dtype=dt, device="cuda")
    v = torch.empty(kv, pages, D, BT, dtype=dt, device="cuda")
    for h in range(kv):
        k[h] = torch.randn(pages * BT, D, device="cuda", generator=g)
        v[h] = torch.randn(pages, D, BT, device="cuda", generator=g).add_(0.25)
    return k, v


def _tables(order, n_tokens, width):
    """Tables of sequences whose pages are taken from `order` one after another."""
    t = torch.full((len(n_tokens), width), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(n_tokens):
        nb = (n + BT - 1) // BT
        t[s, :nb] = order[at:at + nb].int()
        at += nb
    return t


def prepare(case, seed):
    op = case["op"]
    g, cg = _gen(seed), _cpu_gen(seed + 7)
    s = {"op": op}
    kv = case["kv"]
    if op == "prompt":
        dt, heads = _DT[case["dt"]], kv * case["group"]
        s["lq"], s["lk"] = _lens(case)
        tq, tk = sum(s["lq"]), sum(s["lk"])
        if case["fused"] and s["lq"] == s["lk"]:   # slices of a projection's rows: the query heads, then K, then V
            row = _normal(g, tq, heads + 2 * kv, D, dt=dt)
            s["q"], s["k"], s["v"] = row[:, :heads], row[:, heads:heads + kv], row[:, heads + kv:]
            s["v"] += 0.25
        else:
            s["q"] = _normal(g, tq, heads, D, dt=dt)
            s["k"], s["v"] = _normal(g, tk, kv, D, dt=dt), _normal(g, tk, kv, D, dt=dt, mean=0.25)
        s["cu_q"], s["cu_k"] = _i32(_cu(s["lq"])), _i32(_cu(s["lk"]))
        s["out"] = torch.empty(tq, heads, D, dtype=dt, device="cuda")
        s["lse"] = torch.empty(tq, heads, device="cuda")
    elif op == "tree":
        dt, heads, n = _DT[case["dt"]], kv * case["group"], case["seqs"]
        ragged = case["ragged"]
        # ragged lengths are spread evenly below the largest, in no order; the first sequence is the largest
        part = [(i * 0.6180339887) % 1.0 if ragged and i else 1.0 for i in range(n)]
        s["n"] = [int(x * case["tokens"]) for x in part]
        s["nodes"] = [max(1, math.ceil((x * 7) % 1.0 * case["nodes"])) if x < 1 else case["nodes"] for x in part]
        total, blocks = sum(s["nodes"]), sum((x + BT - 1) // BT for x in s["n"])
        s["kcache"], s["vcache_t"] = _pool(g, kv, blocks + 3, dt)
        table = _tables(torch.randperm(blocks + 3, generator=cg), s["n"], (max(s["n"]) + BT - 1) // BT + 2)
        s["parents"] = [int(torch.randint(max(-1, i - 5), i, (1,), generator=cg)) if i else -1 for m in s["nodes"] for i in range(m)]
        s["q"] = _normal(g, total, heads, D, dt=dt)
        s["k"], s["v"] = _normal(g, total, kv, D, dt=dt), _normal(g, total, kv, D, dt=dt, mean=0.25)
        s["dev_parents"], s["cu"], s["n_tokens"], s["table"] = _i32(s["parents"]), _i32(_cu(s["nodes"])), _i32(s["n"]), table.cuda()
        s["out"] = torch.empty(total, heads, D, dtype=dt, device="cuda")
        s["lse"] = torch.empty(total, heads, device="cuda")
    elif op == "commit":
        dt, n = _DT[case["dt"]], case["seqs"]
        whole = n == 1   # a prompt's rows as they come; otherwise the accepted nodes of a tree
        s["n"] = [case["tokens"] - (17 * i) % (case["tokens"] // 2 + 1) for i in range(n)]
        s["nodes"] = [case["nodes"]] * n
        took = [m if whole else int(torch.randint(0, m + 1, (1,), generator=cg)) for m in s["nodes"]]
        rows = [torch.randperm(m, generator=cg)[:t].sort().values + i * case["nodes"] for i, (m, t) in enumerate(zip(s["nodes"], took))]
        s["took"], s["rows"] = took, None if whole else torch.cat(rows).int().cuda()
        total = sum(s["nodes"])
        s["k"], s["v"] = _normal(g, total, kv, D, dt=dt), _normal(g, total, kv, D, dt=dt, mean=0.25)
        s["kcache"], s["vcache_t"] = _pool(g, kv, case["pages"], dt)
        width = max((a + b) // BT for a, b in zip(s["n"], s["nodes"])) + 2
        s["table"] = _tables(torch.randperm(case["pages"], generator=cg), s["n"], width).cuda()
        s["cu"], s["n_tokens"], s["add"], s["keep"] = _i32(_cu(took)), _i32(s["n"]), _i32(took), _i32(s["n"])
    elif op == "fork":
        p, w = case["parents"], case["ways"]
        n = [max(1, case["tokens"] - 29 * i) for i in range(p)]
        s["kcache"], s["vcache_t"] = _pool(g, kv, case["pages"], torch.bfloat16)
        order = torch.randperm(case["pages"], generator=cg)
        old = [1 + (13 * i) % (2 * BT) for i in range(p * w)]   # the children of the step before, dropped in this one
        s["table"] = _tables(order, n + old, max(n) // BT + 3).cuda()
        s["n_tokens"] = _i32(n + old)
        s["keep"] = _i32([-1] * p + [0] * (p * w))
        s["src"], s["dst"] = _i32([i // w for i in range(p * w)]), _i32([p + i for i in range(p * w)])
        s["add"] = _i32([1] * (p + p * w))
        s["kblk"] = _normal(g, case["pages"], D, dt=torch.bfloat16)
    else:
        n, pages = case["seqs"], case["pages"]
        s["kcache"], s["vcache_t"] = _pool(g, kv, pages, torch.bfloat16)
        s["kblk"] = _normal(g, pages, D, dt=torch.bfloat16)
        live = max(1, int(pages * case["live"]))
        shared = live // 8 // n   # each sequence begins with the first one's pages
        each = max(1, (live - shared) // n)
        order = torch.randperm(pages, generator=cg)
        table = torch.full((n, shared + each + 1), -1, dtype=torch.int32)
        for i in range(n):
            table[i, :shared] = order[:shared].int()
            mine = order[shared + i * each:shared + (i + 1) * each].int()
            table[i, shared:shared + mine.numel()] = mine
        s["table"] = table.cuda()
        s["table_out"] = torch.empty_like(s["table"])
    if op in ("commit", "fork", "compact"):
        pages = case["pages"]
        held = s["table"].cpu()
        s["refs"] = torch.bincount(held[held >= 0].long(), minlength=pages).int().cuda()
        rows = s["table"].shape[0]
        if op != "compact":
            s["new_tokens"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        moves = pages // 2 if op == "compact" else rows
        s["copy_src"], s["copy_dst"] = (torch.empty(moves, dtype=torch.int32, device="cuda") for _ in "sd")
        if op == "compact":
            s["refs_out"] = torch.empty_like(s["refs"])
    if own:
        from sparse_attention_kv_gb300 import qsa
        if op in ("prompt", "tree"):
            s["ws"] = qsa.alloc_attention_workspace(s["q"].shape[0], s["q"].shape[1], kv)
        else:
            s["ws"] = qsa.alloc_pages_workspace(s["table"].shape[0], case["pages"])
    return s


# ------------------------------------------------------------------ one pass

def _softmax_rows(z, v):
    """(output, log-sum-exp) of logits z [.., rows, keys] (-inf: unseen) over values v [.., keys, D]."""
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total > 0, total, 1.0), (m + torch.log(total)).squeeze(-1)


def _prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    heads, kv = q.shape[1], k.shape[1]
    out, lse = torch.zeros(q.shape, dtype=q.dtype, device=q.device), torch.full(q.shape[:2], -math.inf, device=q.device)
    qa = ka = 0
    for lq, lk in zip(s["lq"], s["lk"]):
        keys = k[ka:ka + lk].float().transpose(0, 1)                                        # [kv, lk, D]
        vals = v[ka:ka + lk].float().transpose(0, 1)
        step = max(1, min(lq, (1 << 29) // (heads * max(1, lk))))
        for a in range(0, lq, step):
            b = min(a + step, lq)
            seen = max(0, lk - lq + b)
            if seen == 0:
                continue
            x = q[qa + a:qa + b].float().view(b - a, kv, heads // kv, D).permute(1, 2, 0, 3)  # [kv, group, rows, D]
            x = x.reshape(kv, -1, D)
            z = (x @ keys[:, :seen].transpose(-1, -2)) * D ** -0.5
            z = z.view(kv, heads // kv, b - a, seen)
            limit = lk - lq + 1 + torch.arange(a, b, device=q.device)
            z.masked_fill_(torch.arange(seen, device=q.device)[None] >= limit[:, None], -math.inf)
            o, l = _softmax_rows(z.view(kv, -1, seen), vals[:, :seen])
            out[qa + a:qa + b] = o.view(kv, heads // kv, b - a, D).permute(2, 0, 1, 3).reshape(b - a, heads, D).to(q.dtype)
            lse[qa + a:qa + b] = l.view(kv, heads // kv, b - a).permute(2, 0, 1).reshape(b - a, heads)
        qa, ka = qa + lq, ka + lk
    return {"out": out, "lse": lse}


def _ancestors(parents):
    """[n, n] truth values: node i sees node j when j is i or an ancestor of i."""
    n = len(parents)
    sees = [[False] * n for _ in range(n)]
    for i, p in enumerate(parents):
        if p >= 0:
            sees[i] = list(sees[p])
        sees[i][i] = True
    return torch.tensor(sees, device="cuda")


def _tree(s):
    q, k, v = s["q"], s["k"], s["v"]
    heads, kv = q.shape[1], k.shape[1]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=q.device)
    a = 0
    for i, (n, m) in enumerate(zip(s["n"], s["nodes"])):
        b = a + m
        pages = s["table"][i, :(n + BT - 1) // BT].long()
        past_k = s["kcache"].view(kv, -1, BT, D)[:, pages].reshape(kv, -1, D)[:, :n].float()
        past_v = s["vcache_t"][:, pages].transpose(-1, -2).reshape(kv, -1, D)[:, :n].float()
        keys = torch.cat((past_k, k[a:b].float().transpose(0, 1)), 1)
        vals = torch.cat((past_v, v[a:b].float().transpose(0, 1)), 1)
        x = q[a:b].float().view(m, kv, heads // kv, D).permute(1, 2, 0, 3).reshape(kv, -1, D)
        z = ((x @ keys.transpose(-1, -2)) * D ** -0.5).view(kv, heads // kv, m, n + m)
        z[..., n:].masked_fill_(~_ancestors(s["parents"][a:b]), -math.inf)
        o, l = _softmax_rows(z.view(kv, -1, n + m), vals)
        out[a:b] = o.view(kv, heads // kv, m, D).permute(2, 0, 1, 3).reshape(m, heads, D).to(q.dtype)
        lse[a:b] = l.view(kv, heads // kv, m).permute(2, 0, 1).reshape(m, heads)
        a = b
    return {"out": out, "lse": lse}


def _release(table, n_tokens, refs, keep):
    at = torch.arange(table.shape[1], device="cuda")
    drop = (keep[:, None] >= 0) & (at[None] >= (keep[:, None] + BT - 1) // BT) & (table >= 0)
    refs.index_add_(0, torch.where(drop, table, 0).reshape(-1).long(), -drop.reshape(-1).int())
    table.masked_fill_(drop, -1)
    n_tokens.copy_(torch.where(keep >= 0, torch.minimum(keep, n_tokens), n_tokens))


def _fork(table, n_tokens, refs, src, dst):
    nb = (n_tokens + BT - 1) // BT
    rows = table[src.long()]
    rows = torch.where(torch.arange(table.shape[1], device="cuda")[None] < nb[src.long()][:, None], rows, -1)
    table[dst.long()] = rows
    n_tokens[dst.long()] = n_tokens[src.long()]
    refs.index_add_(0, rows.clamp(min=0).reshape(-1).long(), (rows >= 0).int().reshape(-1))


def _reserve(table, n_tokens, refs, add, new_tokens, copy_src, copy_dst):
    """Pages for add[s] more tokens, the lowest free ones first, sequence by sequence; a shared last page is replaced."""
    at = torch.arange(table.shape[1], device="cuda")[None]
    n = n_tokens[:, None]
    missing = (at >= (n + BT - 1) // BT) & (at < (n + add[:, None] + BT - 1) // BT) & (table < 0)
    last = torch.where(n_tokens % BT > 0, table.gather(1, (n_tokens // BT).clamp(max=table.shape[1] - 1)[:, None].long())[:, 0], -1)
    writes = (add > 0) & (last >= 0)
    earlier = (writes[None] & writes[:, None] & (last[None] == last[:, None])).tril(-1).sum(1)
    copies = writes & (refs[last.clamp(min=0).long()] - earlier > 1)
    missing |= copies[:, None] & (at == n // BT)
    free = torch.nonzero(refs == 0)[:, 0]
    rank = (missing.reshape(-1).cumsum(0) - 1).view_as(missing)
    table.copy_(torch.where(missing, free[rank.clamp(min=0, max=max(0, free.numel() - 1))].int(), table))
    refs.index_add_(0, torch.where(missing, table, 0).reshape(-1).long(), missing.reshape(-1).int())
    refs.index_add_(0, last.clamp(min=0).long(), -copies.int())
    new_tokens.copy_(n_tokens + add)
    copy_src.copy_(torch.where(copies, last, -1))
    copy_dst.copy_(torch.where(copies, table.gather(1, (n_tokens // BT).clamp(max=table.shape[1] - 1)[:, None].long())[:, 0], -1))


def _copy(arrays, src, dst):
    take = src >= 0
    a, b = src[take].long(), dst[take].long()
    for x, dim in arrays:
        x.index_copy_(dim, b, x.index_select(dim, a))


def _append(s):
    kv = s["k"].shape[1]
    lens = torch.tensor(s["took"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device="cuda"), lens, output_size=sum(s["took"]))
    pos = s["n_tokens"].long()[seq] + torch.arange(seq.numel(), device="cuda") - s["cu"].long()[seq]
    page = s["table"][seq, pos // BT].long()
    rows = torch.arange(seq.numel(), device="cuda") if s["rows"] is None else s["rows"].long()
    s["kcache"].view(kv, -1, BT, D)[:, page, pos % BT] = s["k"][rows].transpose(0, 1)
    s["vcache_t"].transpose(-1, -2)[:, page, pos % BT] = s["v"][rows].transpose(0, 1)


def _compact(table, refs, table_out, refs_out, copy_src, copy_dst):
    pages = refs.numel()
    at = torch.arange(pages, device="cuda")
    live = refs > 0
    n = live.sum()
    holes, high = torch.nonzero(~live & (at < n))[:, 0], torch.nonzero(live & (at >= n))[:, 0]
    to = at.clone()
    to[high] = holes
    refs_out.zero_()
    refs_out[to[live]] = refs[live]
    table_out.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), -1))
    copy_src.fill_(-1)
    copy_dst.fill_(-1)
    copy_src[:high.numel()] = high.int()
    copy_dst[:high.numel()] = holes.int()


def _paged(s):
    kv = s["kcache"].shape[0]
    return s["kcache"].view(kv, -1, BT, D), s["vcache_t"]


def run(s):
    op = s["op"]
    if own:
        from sparse_attention_kv_gb300 import qsa
        if op == "prompt":
            qsa.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], s["lse"], ws=s["ws"])
        elif op == "tree":
            qsa.tree_attention(s["q"], s["k"], s["v"], s["dev_parents"], s["cu"], max(s["nodes"]), s["kcache"], s["vcache_t"],
                               s["table"], s["n_tokens"], s["out"], s["lse"], ws=s["ws"])
        elif op == "commit":
            qsa.pages_release(s["table"], s["n_tokens"], s["refs"], s["keep"], ws=s["ws"])
            qsa.pages_reserve(s["table"], s["n_tokens"], s["refs"], s["add"], s["new_tokens"], s["copy_src"], s["copy_dst"], ws=s["ws"])
            qsa.pages_append(s["k"], s["v"], s["table"], s["n_tokens"], s["cu"], s["kcache"], s["vcache_t"], rows=s["rows"], ws=s["ws"])
        elif op == "fork":
            qsa.pages_release(s["table"], s["n_tokens"], s["refs"], s["keep"], ws=s["ws"])
            qsa.pages_fork(s["table"], s["n_tokens"], s["refs"], s["src"], s["dst"], ws=s["ws"])
            qsa.pages_reserve(s["table"], s["n_tokens"], s["refs"], s["add"], s["new_tokens"], s["copy_src"], s["copy_dst"], ws=s["ws"])
            qsa.pages_copy([*_paged(s), s["kblk"]], s["copy_src"], s["copy_dst"], ws=s["ws"])
        else:
            qsa.pages_compact(s["table"], s["refs"], s["table_out"], s["refs_out"], s["copy_src"], s["copy_dst"], ws=s["ws"])
            qsa.pages_copy([*_paged(s), s["kblk"]], s["copy_src"], s["copy_dst"], ws=s["ws"])
    elif op == "prompt":
        return _prompt(s)
    elif op == "tree":
        return _tree(s)
    elif op == "commit":
        _release(s["table"], s["n_tokens"], s["refs"], s["keep"])
        _reserve(s["table"], s["n_tokens"], s["refs"], s["add"], s["new_tokens"], s["copy_src"], s["copy_dst"])
        _append(s)
    elif op == "fork":
        _release(s["table"], s["n_tokens"], s["refs"], s["keep"])
        _fork(s["table"], s["n_tokens"], s["refs"], s["src"], s["dst"])
        _reserve(s["table"], s["n_tokens"], s["refs"], s["add"], s["new_tokens"], s["copy_src"], s["copy_dst"])
        _copy([(x, 1) for x in _paged(s)] + [(s["kblk"], 0)], s["copy_src"], s["copy_dst"])
    else:
        _compact(s["table"], s["refs"], s["table_out"], s["refs_out"], s["copy_src"], s["copy_dst"])
        _copy([(x, 1) for x in _paged(s)] + [(s["kblk"], 0)], s["copy_src"], s["copy_dst"])
    names = {"prompt": ("out", "lse"), "tree": ("out", "lse"),
             "commit": ("table", "refs", "n_tokens", "new_tokens", "kcache", "vcache_t"),
             "fork": ("table", "refs", "n_tokens", "new_tokens", "copy_src", "copy_dst", "kcache", "vcache_t", "kblk"),
             "compact": ("table_out", "refs_out", "copy_src", "copy_dst", "kcache", "vcache_t", "kblk")}[op]
    return {n: s[n] for n in names}


# ------------------------------------------------------------------ what a pass cannot do without

def _moved(case):
    """Pages that a compaction moves, on average: the live ones behind the live number of pages."""
    n, live = case["seqs"], max(1, int(case["pages"] * case["live"]))
    shared = live // 8 // n
    live = shared + n * max(1, (live - shared) // n)
    return max(0, live * (1 - live / case["pages"]))


def work(case):
    op, kv = case["op"], case["kv"]
    page = kv * 4 * BT * D
    if op == "prompt":
        lq, lk = _lens(case)
        heads = kv * case["group"]
        # rows with n, n - 1, ... keys, down to none
        pairs = sum((min(a, b) * b - min(a, b) * (min(a, b) - 1) // 2) for a, b in zip(lq, lk))
        b = 2 * D * (2 * sum(lq) * heads + 2 * sum(lk) * kv) + 4 * sum(lq) * heads + 8 * (len(lq) + 1)
        return {"bytes": b, "flops": 4 * D * heads * pairs}
    if op == "tree":
        heads, r = kv * case["group"], (0.5 if case["ragged"] else 1.0)
        n, m = case["tokens"] * (1 + (case["seqs"] - 1) * r), case["nodes"] * (1 + (case["seqs"] - 1) * r)
        seen = n / case["seqs"] + 2
        return {"bytes": 4 * D * kv * (n + m) + m * heads * (4 * D + 4) + 4 * n / BT, "flops": 4 * D * heads * m * seen}
    if op == "commit":
        rows = case["nodes"] * (1 if case["seqs"] == 1 else case["seqs"] / 2)
        return {"bytes": 8 * D * kv * rows + 4 * case["pages"], "flops": 0}
    if op == "fork":
        rows = case["parents"] * (1 + case["ways"])
        return {"bytes": 2 * (page + 2 * D) * case["parents"] * case["ways"] + 8 * rows * (case["tokens"] // BT + 1) + 4 * case["pages"],
                "flops": 0}
    return {"bytes": 2 * (page + 2 * D) * _moved(case) + 16 * case["pages"], "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits

def _attended(q, keys, vals, sees):
    """Rows q [m, heads, D] over keys, vals [n, kv, D] where sees [m, n]; all in float64."""
    m, heads, _ = q.shape
    kv = keys.shape[1]
    out, lse = torch.zeros_like(q), torch.full((m, heads), -math.inf, dtype=torch.float64, device=q.device)
    some = sees.any(1)
    for h in range(heads):
        z = torch.einsum("md,nd->mn", q[:, h], keys[:, h // (heads // kv)]) / math.sqrt(D)
        z.masked_fill_(~sees, -math.inf)
        lse[:, h] = torch.logsumexp(z, 1)
        out[some, h] = torch.softmax(z[some], 1) @ vals[:, h // (heads // kv)]
    return out, lse


def exact(case, seed):
    op = case["op"]
    if op not in ("prompt", "tree"):   # whole numbers and moved bytes only
        return None
    s = prepare(case, seed)
    q, k, v = (s[x].double() for x in "qkv")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    if op == "prompt":
        a = c = 0
        for lq, lk in zip(s["lq"], s["lk"]):
            for r in range(0, lq, 2048):
                e = min(lq, r + 2048)
                n = max(1, min(lk, lk - lq + e))   # no row of this piece sees more
                if lk == 0:
                    out[a + r:a + e], lse[a + r:a + e] = 0.0, -math.inf
                    continue
                sees = torch.arange(n, device="cuda")[None] <= (torch.arange(r, e, device="cuda") + lk - lq)[:, None]
                out[a + r:a + e], lse[a + r:a + e] = _attended(q[a + r:a + e], k[c:c + n], v[c:c + n], sees)
            a, c = a + lq, c + lk
        return {"out": out, "lse": lse}
    a = 0
    for i, (n, m) in enumerate(zip(s["n"], s["nodes"])):
        tokens = torch.arange(n, device="cuda")
        page = s["table"][i].long()[tokens // BT]
        keys = torch.cat((s["kcache"][:, page * BT + tokens % BT].double().transpose(0, 1), k[a:a + m]))
        vals = torch.cat((s["vcache_t"][:, page, :, tokens % BT].double().reshape(n, v.shape[1], D), v[a:a + m]))
        line = []
        for j, p in enumerate(s["parents"][a:a + m]):   # walk up from each node
            up = {j}
            while p >= 0:
                up.add(p)
                p = s["parents"][a + p]
            line.append([x in up for x in range(m)])
        sees = torch.cat((torch.ones(m, n, dtype=torch.bool, device="cuda"), torch.tensor(line, device="cuda")), 1)
        out[a:a + m], lse[a:a + m] = _attended(q[a:a + m], keys, vals, sees)
        a += m
    return {"out": out, "lse": lse}
