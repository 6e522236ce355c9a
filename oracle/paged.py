"""Plain definition of the paged 16-bit cache and of the dense attentions over it, in 64 bits: what the
library's calls do to tables, references and pages, row by row, and the softmax attention of packed
prompts and of drafted trees.  Test infrastructure only; it shares no code with the library."""
import math

import torch

BT = 64
D = 128


# ------------------------------------------------------------------ attention

def attended(q, k, v, sees, scale):
    """(out, lse, mass, logit) of rows q [m, heads, D] over k, v [n, kv, D] (float64) where sees [m, n]: mass is
    the output over |v|, logit the largest scale * sum |q||k| a row meets among what it sees."""
    m, heads, _ = q.shape
    group = heads // k.shape[1]
    out, mass = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((m, heads), -math.inf, dtype=torch.float64, device=q.device)
    logit = torch.zeros_like(lse)
    some = sees.any(1)
    if not bool(some.any()):
        return out, lse, mass, logit
    for h in range(heads):
        kh, vh = k[:, h // group], v[:, h // group]
        seen = sees[some]
        z = (scale * (q[some, h] @ kh.T)).masked_fill(~seen, -math.inf)
        lse[some, h] = torch.logsumexp(z, 1)
        p = torch.softmax(z, 1)
        use = seen[:, :, None]
        if bool(torch.isfinite(vh).all()):
            out[some, h], mass[some, h] = p @ vh, p @ vh.abs()
        else:   # what is not seen is not touched, not even by a weight of zero
            out[some, h] = torch.where(use, p[:, :, None] * vh[None], 0.0).sum(1)
            mass[some, h] = torch.where(use, p[:, :, None] * vh[None].abs(), 0.0).sum(1)
        logit[some, h] = (scale * (q[some, h].abs() @ kh.abs().T)).masked_fill(~seen, 0.0).amax(1)
    return out, lse, mass, logit


def prompt(q, k, v, lq, lk, scale):
    """Packed causal attention; query i of a sequence sees its first lk - lq + i + 1 keys."""
    parts, a, c = [], 0, 0
    for m, n in zip(lq, lk):
        at = torch.arange(m, device=q.device)[:, None] + n - m
        sees = torch.arange(n, device=q.device)[None] <= at
        parts.append(attended(q[a:a + m], k[c:c + n], v[c:c + n], sees, scale))
        a, c = a + m, c + n
    return [torch.cat(x) for x in zip(*parts)]


def ancestors(parents):
    """[n][n]: node i sees node j when j is i or above it; a parent that is not before its node counts as none."""
    sees = []
    for i, p in enumerate(parents):
        row = list(sees[p]) if 0 <= p < i else [False] * len(parents)
        row[i] = True
        sees.append(row)
    return sees


def paged_rows(kcache, vcache_t, pages, n):
    """The first n token rows (K and V, [n, kv, D]) of a sequence whose pages are listed; None where a page is no page."""
    kv, total = kcache.shape[0], vcache_t.shape[1]
    t = torch.arange(n, device=kcache.device)
    page = torch.as_tensor(pages, device=kcache.device).long()[t // BT]
    ok = (page >= 0) & (page < total)
    page = page.clamp(0, total - 1)
    k = kcache.view(kv, total, BT, D)[:, page, t % BT].transpose(0, 1)
    return k, vcache_t[:, page, :, t % BT].reshape(n, kv, D), ok


def tree(q, k, v, parents, nodes, kcache, vcache_t, table, n_tokens, scale):
    """Drafted trees over pages (float64 rows and pools; parents, nodes, table, n_tokens as lists)."""
    parts, a = [], 0
    for s, m in enumerate(nodes):
        pk, pv, ok = paged_rows(kcache, vcache_t, table[s], n_tokens[s])
        sees = torch.tensor(ancestors(parents[a:a + m]), dtype=torch.bool, device=q.device).view(m, m)
        sees = torch.cat((ok[None].expand(m, -1), sees), 1)
        parts.append(attended(q[a:a + m], torch.cat((pk, k[a:a + m])), torch.cat((pv, v[a:a + m])), sees, scale))
        a += m
    return [torch.cat(x) for x in zip(*parts)]


# ------------------------------------------------------------------ pages

class Pool:
    """Tables and references as lists; every call as qsa.h words it, one row after another."""

    def __init__(self, table, n_tokens, refs):
        self.table, self.n, self.refs = [list(r) for r in table], list(n_tokens), list(refs)
        self.flags = set()

    def _page(self, p):
        return 0 <= p < len(self.refs)

    def _drop(self, p):
        if self.refs[p] > 0:
            self.refs[p] -= 1
        else:
            self.flags.add("id")

    def fork(self, src, dst):
        rows, width = len(self.table), len(self.table[0])
        for i, (a, b) in enumerate(zip(src, dst)):
            if a == -1 and b == -1:
                continue
            if not (0 <= a < rows and 0 <= b < rows) or b in dst[:i] or b in src or self.n[b] > 0:
                self.flags.add("id")
                continue
            for p in self.table[b]:
                if self._page(p):
                    self._drop(p)
            n = min(max(self.n[a], 0), BT * width)
            if n != self.n[a]:
                self.flags.add("clamp")
            self.table[b] = [-1] * width
            for j in range((n + BT - 1) // BT):
                p = self.table[a][j]
                if self._page(p):
                    self.table[b][j] = p
                    self.refs[p] += 1
                else:
                    self.flags.add("id")
            self.n[b] = n

    def release(self, keep):
        for s, left in enumerate(keep):
            if left < 0:
                continue
            for j in range((left + BT - 1) // BT, len(self.table[s])):
                p = self.table[s][j]
                if self._page(p):
                    self._drop(p)
                    self.table[s][j] = -1
                elif p != -1:
                    self.flags.add("id")
            self.n[s] = min(self.n[s], left)

    def reserve(self, add):
        """-> (new_tokens, copy_src, copy_dst)"""
        width = len(self.table[0])
        free = [p for p, r in enumerate(self.refs) if r == 0]
        held = list(self.refs)                       # before the call
        new, cs, cd = list(self.n), [-1] * len(self.n), [-1] * len(self.n)
        asked, writers = 0, {}
        for s, (n, more) in enumerate(zip(self.n, add)):
            if more < 0:
                self.flags.add("clamp")
                more = 0
            if n < 0 or n + more > BT * width:
                self.flags.add("clamp")
                continue
            past = [self.table[s][j] for j in range((n + BT - 1) // BT, (n + more + BT - 1) // BT)] if more > 0 else []
            if any(self._page(p) and held[p] > 1 for p in past):
                self.flags.add("id")             # another row's page behind the tokens
                continue
            want = []
            shared = keeps = False
            if more > 0:
                if n % BT:
                    p = self.table[s][n // BT]
                    if not self._page(p):
                        self.flags.add("id")
                        want.append(n // BT)
                    else:
                        before = writers.get(p, 0)
                        writers[p] = before + 1
                        shared = held[p] > 1 and held[p] - before > 1
                        keeps = held[p] > 1 and not shared
                        if shared:
                            want.append(n // BT)
                for j in range((n + BT - 1) // BT, (n + more + BT - 1) // BT):
                    if not self._page(self.table[s][j]):
                        if self.table[s][j] != -1:
                            self.flags.add("id")
                        want.append(j)
            asked += len(want)
            if asked > len(free) and (want or keeps):
                self.flags.add("pages")
                continue
            mine = free[asked - len(want):asked]
            if shared:
                cs[s], cd[s] = self.table[s][n // BT], mine[0]
                self.refs[cs[s]] -= 1
            for j, p in zip(want, mine):
                self.table[s][j] = p
                self.refs[p] = 1
            new[s] = n + more
        return new, cs, cd

    def compact(self):
        """-> (table, refs, copy_src, copy_dst)"""
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] <= 0]
        high = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = {p: p for p in range(live)}
        to.update(zip(high, holes))
        refs = [0] * len(self.refs)
        for p, r in enumerate(self.refs):
            if r > 0:
                refs[to[p]] = r
        table = []
        for row in self.table:
            table.append([to.get(p, -1) for p in row])
            if any(p not in to and p != -1 for p in row):
                self.flags.add("id")
        pad = [-1] * (len(self.refs) // 2 - len(high))
        return table, refs, high + pad, holes + pad

    def append(self, k, v, first, cu, kcache, vcache_t, rows=None, end=None):
        """Rows of k, v [n, kv, D] (tensors) into the pools, in place; none at or past a row's end."""
        width, pages = len(self.table[0]), kcache.shape[1] // BT
        entries = k.shape[0] if rows is None else len(rows)
        for s in range(len(self.table)):
            if not 0 <= cu[s] <= cu[s + 1] <= entries:
                self.flags.add("clamp")
            if cu[s + 1] < cu[s]:            # neither this row nor the ones behind it
                break
            c0, c1 = (min(max(c, 0), entries) for c in cu[s:s + 2])
            for e in range(c0, c1):
                r, pos = (e if rows is None else rows[e]), first[s] + e - c0
                if pos < 0 or pos >= BT * width:
                    self.flags.add("clamp")
                    continue
                if end is not None and pos >= end[s]:
                    continue
                p = self.table[s][pos // BT]
                if not 0 <= p < pages:
                    self.flags.add("id")
                    continue
                if not 0 <= r < k.shape[0]:
                    if r != -1:
                        self.flags.add("id")
                    continue
                kcache[:, p * BT + pos % BT] = k[r]
                vcache_t[:, p, :, pos % BT] = v[r]
