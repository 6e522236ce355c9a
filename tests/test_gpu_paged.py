"""The pages of the 16-bit cache on the GPU against their definition, and a generation over them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from oracle import paged  # noqa: E402
from sparse_attention_kv_gb300 import qsa  # noqa: E402

from .paged_cases import check_attention, cu, i32, normal, random_parents, random_pool  # noqa: E402

BITS = {"id": qsa.FLAG_BAD_ID, "clamp": qsa.FLAG_NBLOCKS_CLAMPED, "pages": qsa.FLAG_NO_PAGES}


class Both:
    """A pool on the GPU beside its definition; every call goes to both, and all state is compared."""

    def __init__(self, table, n_tokens, refs, stride=None):
        self.pool = paged.Pool(table, n_tokens, refs)
        rows, width = len(table), len(table[0])
        wide = torch.full((rows, stride or width), 77, dtype=torch.int32, device="cuda")
        wide[:, :width] = i32(table)
        self.wide, self.table = wide, wide[:, :width]
        self.n, self.refs = i32(n_tokens), i32(refs)
        self.ws = qsa.alloc_pages_workspace(rows, len(refs))

    def check(self):
        p = self.pool
        assert self.table.tolist() == p.table
        assert self.n.tolist() == p.n and self.refs.tolist() == p.refs
        assert (self.wide[:, self.table.shape[1]:] == 77).all()
        want = 0
        for f in p.flags:
            want |= BITS[f]
        assert qsa.read_flags(self.ws) == want
        p.flags.clear()

    def fork(self, src, dst):
        qsa.pages_fork(self.table, self.n, self.refs, i32(src), i32(dst), ws=self.ws)
        self.pool.fork(src, dst)
        self.check()

    def release(self, keep):
        qsa.pages_release(self.table, self.n, self.refs, i32(keep), ws=self.ws)
        self.pool.release(keep)
        self.check()

    def reserve(self, add):
        rows = len(add)
        new, cs, cd = (torch.full((rows,), 99, dtype=torch.int32, device="cuda") for _ in range(3))
        qsa.pages_reserve(self.table, self.n, self.refs, i32(add), new, cs, cd, ws=self.ws)
        want = self.pool.reserve(add)
        assert [new.tolist(), cs.tolist(), cd.tolist()] == [list(x) for x in want]
        self.check()
        return new, cs, cd

    def compact(self, in_place):
        pages = self.refs.numel()
        cs, cd = (torch.full((pages // 2,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
        t, r = (self.table, self.refs) if in_place else (torch.empty_like(self.wide)[:, :self.table.shape[1]], torch.empty_like(self.refs))
        qsa.pages_compact(self.table, self.refs, t, r, cs, cd, ws=self.ws)
        table, refs, src, dst = self.pool.compact()
        assert t.tolist() == table and r.tolist() == refs
        assert cs.tolist() == src and cd.tolist() == dst
        if in_place:
            self.pool.table, self.pool.refs = table, refs
        self.check()
        return cs, cd


def _random(seed, rows, width, pages, fill=0.6):
    """Tables of random lengths, some sharing another's first pages, with reserved pages behind some."""
    rng = np.random.default_rng(seed)
    order = rng.permutation(pages).tolist()
    table, n, refs = [], [], [0] * pages
    for s in range(rows):
        row = []
        if s and rng.random() < 0.5:
            of = int(rng.integers(0, s))
            full = [p for p in table[of] if p >= 0]
            row = full[:int(rng.integers(0, len(full) + 1))]
        more = int(rng.integers(0, max(1, int(fill * width)) + 1))
        while more and order and len(row) < width:
            row.append(order.pop())
            more -= 1
        hi = 64 * len(row)
        n.append(int(rng.integers(max(0, hi - 130), hi + 1)))
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (width - len(row)))
    return table, n, refs


SIZES = [(1, 1, 1), (1, 5, 3), (3, 4, 20), (17, 9, 200), (64, 40, 3000), (300, 70, 5000), (5, 2050, 9000)]


@pytest.mark.parametrize("rows,width,pages", SIZES)
def test_release_and_fork_match_the_definition(rows, width, pages):
    rng = np.random.default_rng(rows)
    b = Both(*_random(rows, rows, width, pages), stride=width + 3)
    keep = rng.integers(-1, 64 * width, size=rows)
    keep[rng.random(rows) < 0.4] = 0
    b.release(keep.tolist())
    empty = [s for s in range(rows) if b.pool.n[s] == 0]
    full = [s for s in range(rows) if b.pool.n[s] > 0]
    if full and empty:
        b.fork([int(rng.choice(full)) for _ in empty], empty)
    b.release([-1] * rows)
    b.release([2 ** 31 - 1] * rows)
    b.release([0] * rows)
    assert not any(b.pool.refs)


@pytest.mark.parametrize("rows,width,pages", SIZES)
@pytest.mark.parametrize("kind", ["ones", "random", "many"])
def test_reserve_matches_the_definition(rows, width, pages, kind):
    rng = np.random.default_rng(rows + len(kind))
    b = Both(*_random(rows + 1, rows, width, pages))
    for _ in range(3):
        room = [64 * width - x for x in b.pool.n]
        if kind == "ones":
            add = [min(1, r) for r in room]
        else:
            add = [int(rng.integers(0, min(r, 200 if kind == "random" else r) + 1)) for r in room]
        new, _, _ = b.reserve(add)
        b.n.copy_(new)
        b.pool.n = new.tolist()


def test_reserve_settles_shared_pages():
    """Rows that share a partial page and write: all but the last one copy, or all when someone else holds it too."""
    table = [[3, 7, -1], [3, 7, -1], [3, 7, -1], [3, 7, -1], [9, -1, -1]]
    refs = [0] * 12
    refs[3], refs[7], refs[9] = 4, 4, 1
    b = Both(table, [100, 100, 100, 100, 64], refs)
    new, cs, cd = b.reserve([1, 0, 30, 5, 0])           # row 1 does not write
    assert cs.tolist() == [7, -1, 7, 7, -1] and cd.tolist() == [0, -1, 1, 4, -1]
    b = Both(table, [100, 100, 100, 100, 64], refs)
    new, cs, cd = b.reserve([1, 1, 1, 1, 1])
    assert cs.tolist() == [7, 7, 7, -1, -1] and b.table[3].tolist() == [3, 7, -1] and b.table[4].tolist() == [9, 4, -1]
    b = Both(table, [128, 128, 128, 128, 64], refs)     # whole pages are never written again
    _, cs, _ = b.reserve([1] * 5)
    assert cs.tolist() == [-1] * 5


@pytest.mark.parametrize("behind", [1, 2, 3, 40, 128, 129, 2000])
@pytest.mark.parametrize("partial", [0, 1])
def test_reserve_leaves_rows_with_shared_pages_behind_their_tokens(behind, partial):
    """Rows 0 and 1 have the same pages; row 1's length was lowered by hand, by a page and by all of them.  Released, it is served."""
    width, n = behind + 6, 64 * (behind + 3)
    shared = list(range(behind + 3))
    table = [shared + [-1] * 3, shared + [-1] * 3, [behind + 3] + [-1] * (width - 1), [behind + 4] + [-1] * (width - 1)]
    refs = [2] * (behind + 3) + [1, 1] + [0] * (2 * behind + 20)
    for left in (64 * 3 - partial, n - 64 - partial):
        b = Both(table, [n, left, 64, 1], refs)
        room = n - left
        new, cs, cd = b.reserve([0, room, 70, 1])
        assert new.tolist() == [n, left, 134, 2] and b.table[1].tolist() == table[1]
        b.n.copy_(new)
        b.pool.n = new.tolist()
        b.release([-1, left, -1, -1])
        new, cs, cd = b.reserve([0, room, 1, 1])
        assert new.tolist() == [n, n, 135, 3] and (cs[1] >= 0) == bool(partial)
    b = Both(table, [n, 64, 64, 1], refs)                # reserved pages of its own behind shared ones, and without new tokens
    b.reserve([64, 0, 0, 0])
    b.reserve([1, 1, 1, 1])


def test_reserve_without_enough_pages():
    refs = [1, 1, 0, 1, 0, 2]
    table = [[0, -1, -1], [1, -1, -1], [3, 5, -1], [5, -1, -1]]
    for add in ([1, 1, 1, 1], [64, 64, 64, 0], [65, 0, 0, 10], [0, 129, 1, 1], [-3, 10, 1, 200], [129, 1, 64, 1]):
        Both([list(r) for r in table], [64, 64, 100, 36], refs).reserve(add)
    # a row that would keep a shared page is not served when a row before it could not leave it
    b = Both([[0, 1], [0, -1]], [70, 3], [2, 1])
    b.reserve([10, 1])
    b = Both([[0, -1], [0, -1]], [3, 3], [2])
    new, cs, _ = b.reserve([1, 1])
    assert new.tolist() == [3, 3] and cs.tolist() == [-1, -1]


def test_bad_entries_are_flagged_and_left():
    refs = [1, 1, 0, 1, 0, 0, 0, 0]
    b = Both([[0, 99, -1], [1, -7, -1], [3, 2, -1]], [128, 128, 70], refs)
    b.release([64, 64, 64])                              # page 2 has no reference
    b = Both([[0, 99, -1], [1, -1, -1], [3, -1, -1]], [70, 70, 10], refs)
    b.reserve([1, 1, 100])
    b = Both([[0, -1, -1], [1, -1, -1], [3, -1, -1], [-1] * 3, [-1] * 3], [64, 64, 10, 0, 0], refs)
    for src, dst in (([0, 0], [3, 3]), ([0], [1]), ([9], [3]), ([0], [-1]), ([0], [5]), ([-1, 1], [-1, 4]), ([3, 0], [4, 3])):
        c = Both([list(r) for r in b.pool.table], b.pool.n, b.pool.refs)
        c.fork(src, dst)
    c = Both([[0, -1, -1], [6, 7, -1]], [64, 0], [1, 0, 0, 0, 0, 0, 1, 1])   # reserved pages of an empty row are given back
    c.fork([0], [1])
    c = Both([[0, 6, -1], [5, -1, 99]], [64, 0], refs)   # compaction: entries that name no live page behind the live ones
    c.compact(False)
    c.compact(True)


@pytest.mark.parametrize("bad", [-1, -2, 8, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("at,tokens", [(0, 200), (1, 200), (3, 200), (3, 192), (2, 129), (1, 64)])
def test_fork_of_a_row_with_entries_that_are_no_page(at, tokens, bad):
    """Below the tokens such an entry becomes -1 and is flagged; behind them it is not looked at."""
    table = [[0, 1, 2, 3], [5, -1, -1, -1], [-1] * 4, [7, 7, -1, -1]]
    table[0][at] = bad
    refs = [1, 1, 1, 1, 0, 1, 0, 2]
    if at < 4:
        refs[at] = 0
    b = Both(table, [tokens, 0, 0, 0], refs)
    b.fork([0, -1, 0], [1, -1, 3])
    assert (b.table[1].tolist()[at] == -1) and b.refs[-1] == 0


@pytest.mark.parametrize("n", [257, 2 ** 31 - 1, -1, -2 ** 31, 256, 0])
def test_fork_of_a_row_whose_length_is_out_of_range(n):
    b = Both([[0, 1, 2, 3], [-1] * 4], [n, 0], [1] * 4 + [0])
    b.fork([0], [1])
    assert b.n.tolist() == [n, min(max(n, 0), 256)]


@pytest.mark.parametrize("rows,width,pages", SIZES + [(2, 3, 2), (40, 300, 20_000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_matches_the_definition(rows, width, pages, in_place):
    b = Both(*_random(rows + 5, rows, width, pages), stride=width + 1)
    before = [list(r) for r in b.pool.table]
    pool = torch.arange(pages, device="cuda", dtype=torch.int32)[None, :, None].expand(2, -1, 5).contiguous()
    cs, cd = b.compact(in_place)
    qsa.pages_copy([pool, pool[0, :, 0].clone()], cs, cd, ws=b.ws)
    table = b.table.tolist() if in_place else b.pool.compact()[0]
    for old, new in zip(before, table):                  # every entry still names its page's contents
        for x, y in zip(old, new):
            assert (x < 0 and y < 0) or (pool[:, y] == x).all()
    assert qsa.read_flags(b.ws) == 0


def test_copy_pages():
    g = torch.Generator(device="cuda").manual_seed(1)
    for shape, dt in (((4, 50, 64, 128), torch.bfloat16), ((3, 50, 8704), torch.uint8), ((50, 128), torch.float16), ((50,), torch.float32),
                      ((2, 50, 3), torch.float32)):
        x = torch.randint(0, 100, shape, device="cuda", generator=g).to(dt)
        y = x.clone()
        src, dst = [3, 3, -1, 7, 49, 12], [0, 1, -1, 48, 2, 20]
        ws = qsa.alloc_pages_workspace(1, 50)
        qsa.pages_copy([x], i32(src), i32(dst), ws=ws)
        dim = 1 if len(shape) > 2 else 0
        for a, b in zip(src, dst):
            if a >= 0:
                y.select(dim, b).copy_(y.select(dim, a))
        assert torch.equal(x, y) and qsa.read_flags(ws) == 0
        for a, b in ((50, 1), (1, 50), (-2, 1), (1, -2), (-1, 4), (4, -1)):
            qsa.pages_copy([x], i32([a]), i32([b]), ws=ws)
            assert torch.equal(x, y) and qsa.read_flags(ws) == qsa.FLAG_BAD_ID, (a, b)
        qsa.pages_copy([x], i32([]), i32([]))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv,lens,first", [(1, [1], [0]), (4, [3], [62]), (2, [0, 5, 130], [7, 64, 63]), (3, [1000], [1]),
                                           (2, [64, 64], [0, 128]), (1, [1] * 70, list(range(0, 700, 10)))])
@pytest.mark.parametrize("pick", [False, True])
def test_append_matches_the_definition(kv, lens, first, pick, dt):
    rows = len(lens)
    width = max((f + m + 63) // 64 for f, m in zip(first, lens)) + 1
    pages = sum((f + m + 63) // 64 for f, m in zip(first, lens)) + 4
    rng = np.random.default_rng(kv + rows)
    order = rng.permutation(pages).tolist()
    table = []
    for f, m in zip(first, lens):
        nb = (f + m + 63) // 64
        table.append([order.pop() for _ in range(nb)] + [-1] * (width - nb))
    n = sum(lens)
    source = n + 9 if pick else n
    fused = normal(3, source, 3 * kv, 128, dt=dt)
    k, v = fused[:, kv:2 * kv], fused[:, 2 * kv:]
    pool = paged.Pool(table, first, [0] * pages)
    kc, vc = random_pool(5, kv, pages, dt)
    kw, vw = kc.clone(), vc.clone()
    idx = rng.integers(-1, source, size=n).tolist() if pick else None    # -1: a place left as it was; repeats
    ws = qsa.alloc_pages_workspace(rows, pages)
    qsa.pages_append(k, v, i32(table), i32(first), i32(cu(lens)), kc, vc, rows=None if idx is None else i32(idx), ws=ws)
    pool.append(k, v, first, cu(lens), kw, vw, idx)
    assert torch.equal(kc, kw) and torch.equal(vc, vw)
    assert qsa.read_flags(ws) == 0 and not pool.flags


def test_append_drops_what_has_no_place():
    kv, pages = 2, 6
    k, v = normal(1, 300, kv, 128, dt=torch.bfloat16), normal(2, 300, kv, 128, dt=torch.bfloat16)
    for table, first, lens, idx in (([[0, 1]], [-5], [20], None), ([[0, 1]], [100], [60], None), ([[0, -1]], [60], [9], None),
                                    ([[0, 9]], [60], [9], None), ([[4, 1], [2, 3]], [2 ** 31 - 1, 0], [5, 5], None),
                                    ([[0, 1]], [0], [4], [0, 300, -2, 299]), ([[0, 1]], [-2 ** 31], [9], None)):
        pool, flags = paged.Pool(table, first, [0] * pages), 0
        kc, vc = random_pool(5, kv, pages, torch.bfloat16)
        kw, vw = kc.clone(), vc.clone()
        n = sum(lens)
        kk, vv = (k, v) if idx else (k[:n], v[:n])
        ws = qsa.alloc_pages_workspace(len(table), pages)
        qsa.pages_append(kk, vv, i32(table), i32(first), i32(cu(lens)), kc, vc, rows=i32(idx) if idx else None, ws=ws)
        pool.append(kk, vv, first, cu(lens), kw, vw, idx)
        assert torch.equal(kc, kw) and torch.equal(vc, vw)
        for f in pool.flags:
            flags |= BITS[f]
        assert qsa.read_flags(ws) == flags and flags
    kc, vc = random_pool(5, kv, pages, torch.bfloat16)
    kw, vw = kc.clone(), vc.clone()
    ws = qsa.alloc_pages_workspace(2, pages)
    qsa.pages_append(k[:10], v[:10], i32([[0], [1]]), i32([0, 0]), i32([0, 99, 4]), kc, vc, ws=ws)   # past the entries; a descent
    paged.Pool([[0], [1]], [0, 0], [0] * pages).append(k[:10], v[:10], [0, 0], [0, 10, 10], kw, vw)
    assert torch.equal(kc, kw) and torch.equal(vc, vw) and qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED


@pytest.mark.parametrize("pick", [False, True])
@pytest.mark.parametrize("kv,lens,first,end", [(1, [1], [0], [0]), (1, [1], [0], [1]), (2, [70, 5, 200, 64], [60, 100, 3, 64], [100, 100, 130, 128]),
                                               (3, [130, 130, 130], [1, 1, 1], [-5, 64, 2 ** 31 - 1]), (1, [1] * 300, [63] * 300, [63, 64] * 150)])
def test_append_ends_where_a_row_has_room(kv, lens, first, end, pick):
    rows, dt = len(lens), torch.float16
    width = max((f + m + 63) // 64 for f, m in zip(first, lens))
    table = [list(range(s * width, (s + 1) * width)) for s in range(rows)]
    n, pages = sum(lens), rows * width
    k, v = normal(3, n + 2, kv, 128, dt=dt), normal(4, n + 2, kv, 128, dt=dt)
    idx = np.random.default_rng(rows).integers(0, n + 2, size=n).tolist() if pick else None
    if not pick:
        k, v = k[:n], v[:n]
    kc, vc = random_pool(5, kv, pages, dt)
    kw, vw = kc.clone(), vc.clone()
    pool = paged.Pool(table, first, [1] * pages)
    ws = qsa.alloc_pages_workspace(rows, pages)
    qsa.pages_append(k, v, i32(table), i32(first), i32(cu(lens)), kc, vc, rows=i32(idx) if pick else None, ws=ws, end=i32(end))
    pool.append(k, v, first, cu(lens), kw, vw, idx, end)
    assert torch.equal(kc, kw) and torch.equal(vc, vw) and qsa.read_flags(ws) == 0 and not pool.flags


@pytest.mark.parametrize("captured", [False, True])
def test_a_row_that_found_no_pages_writes_nothing(captured):
    """Rows 1 and 2 are forks of row 0 that went back into its last page; the pool has a page for one of them, then
    for none: who is refused leaves the others' rows as they are, and is served once there is room."""
    kv, pages, rows, dt = 2, 4, 3, torch.bfloat16
    kc, vc, table, n, refs = qsa.alloc_pages(rows, 4, pages, kv)
    ws = qsa.alloc_pages_workspace(rows, pages)
    new, cs, cd, add, cum = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (rows, rows, rows, rows, rows + 1))
    k, v = normal(1, 200, kv, 128, dt=dt), normal(2, 200, kv, 128, dt=dt)

    def step():
        qsa.pages_reserve(table, n, refs, add, new, cs, cd, ws=ws)
        qsa.pages_copy([kc.view(kv, pages, 64, 128), vc], cs, cd, ws=ws)
        qsa.pages_append(k, v, table, n, cum, kc, vc, rows=idx, ws=ws, end=new)
        n.copy_(new)

    def run(lens, picked):
        add.copy_(i32(lens)), cum.copy_(i32(cu(lens)))
        idx.fill_(-1)
        idx[:len(picked)] = i32(picked)
        if graph is None:
            step()
        else:
            graph.replay()
        for s in range(rows):
            if new[s] > before[s]:
                side[s] = [torch.cat((side[s][0], k[picked[sum(lens[:s]):sum(lens[:s + 1])]])),
                           torch.cat((side[s][1], v[picked[sum(lens[:s]):sum(lens[:s + 1])]]))]
        before[:] = n.tolist()
        assert before == [len(x[0]) for x in side]
        for s in range(rows):
            pk, pv, ok = paged.paged_rows(kc, vc, table[s].tolist(), before[s])
            assert ok.all() and torch.equal(pk, side[s][0]) and torch.equal(pv, side[s][1]), s
        return qsa.read_flags(ws)

    idx = torch.full((200,), -1, dtype=torch.int32, device="cuda")
    none = [k[:0], v[:0]]
    side, before, graph = [list(none) for _ in range(rows)], [0] * rows, None
    assert run([120, 0, 0], list(range(120))) == 0
    qsa.pages_fork(table, n, refs, i32([0, 0]), i32([1, 2]), ws=ws)
    qsa.pages_release(table, n, refs, i32([-1, 100, 90]), ws=ws)
    side[1], side[2] = [x[:100] for x in side[0]], [x[:90] for x in side[0]]
    before[:] = [120, 100, 90]
    if captured:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    # pages 2 and 3 are free: row 1 asks for three, row 2 for one behind it
    assert run([0, 150, 5], list(range(155))) == qsa.FLAG_NO_PAGES and before == [120, 100, 90]
    assert run([3, 0, 3], [7, 8, 9, 1, 2, 3]) == 0 and before == [123, 100, 93]            # a page each
    assert run([5, 30, 2], list(range(37))) == qsa.FLAG_NO_PAGES and before == [128, 100, 95]   # rows 0 and 2 need none
    assert refs.tolist() == [3, 1, 1, 1]


@pytest.mark.parametrize("cuts", [[0, 6400, 0, 6400], [6400, 0, 6400, 6400, 0, 99_999], [-9, 64, 0, 6400], [0, 3200, 100, 3300],
                                  [0] * 300 + [6400, 0, 6400], [0, 6400, 0, 6400] + [6400] * 900, [0, 99_999, 6400, 6000, 6400],
                                  [0, 100] + [100] * 254 + [50, 6400], [0, 100] + [100] * 255 + [50, 6400]])
def test_append_stops_where_the_rows_entries_descend(cuts):
    """The rows before a descent of cu_rows are written, the ones behind it, which may take entries again, are not."""
    kv, n, rows = 1, 6400, len(cuts) - 1
    k, v = normal(1, n, kv, 128, dt=torch.bfloat16), normal(2, n, kv, 128, dt=torch.bfloat16)
    lens = [max(0, min(max(b, 0), n) - min(max(a, 0), n)) for a, b in zip(cuts, cuts[1:])]
    at = cu([(m + 63) // 64 for m in lens])              # pages for all of them
    table = [list(range(a, b)) + [-1] * (100 - b + a) for a, b in zip(at, at[1:])]
    kc, vc = random_pool(5, kv, at[-1], torch.bfloat16)
    kw, vw = kc.clone(), vc.clone()
    pool, ws = paged.Pool(table, [0] * rows, [1] * at[-1]), qsa.alloc_pages_workspace(rows, at[-1])
    qsa.pages_append(k, v, i32(table), i32([0] * rows), i32(cuts), kc, vc, ws=ws)
    pool.append(k, v, [0] * rows, cuts, kw, vw)
    assert torch.equal(kc, kw) and torch.equal(vc, vw)
    assert qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED and pool.flags == {"clamp"}


@pytest.mark.parametrize("bad", [0, 255, 256, 599])
def test_append_looks_at_every_row_for_its_flags(bad):
    """600 rows of one token each, one of them with no place: behind the first pages, and without a page of its own."""
    rows, kv = 600, 1
    k, v = normal(1, rows, kv, 128, dt=torch.bfloat16), normal(2, rows, kv, 128, dt=torch.bfloat16)
    first = [3] * rows
    first[bad] = 64
    table = [[p] for p in range(rows)]
    kc, vc = random_pool(5, kv, rows, torch.bfloat16)
    kw, vw = kc.clone(), vc.clone()
    ws = qsa.alloc_pages_workspace(rows, rows)
    qsa.pages_append(k, v, i32(table), i32(first), i32(cu([1] * rows)), kc, vc, ws=ws)
    paged.Pool(table, first, [0] * rows).append(k, v, first, cu([1] * rows), kw, vw)
    assert torch.equal(kc, kw) and torch.equal(vc, vw) and qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED


@pytest.mark.parametrize("captured", [False, True])
def test_a_generation_over_pages(captured):
    """Prompts attended and appended, sequences forked, trees of drafts attended, their accepted nodes appended
    behind copied pages, sequences dropped, the pool compacted: every output against rows kept on the side."""
    kv, group, pages, width, rows = 2, 4, 40, 8, 4
    kc, vc, table, n, refs = qsa.alloc_pages(rows, width, pages, kv)
    ws, aws = qsa.alloc_pages_workspace(rows, pages), qsa.alloc_attention_workspace(400, kv * group, kv)
    new, cs, cd = (torch.empty(rows, dtype=torch.int32, device="cuda") for _ in range(3))
    add, cum = i32([0] * rows), i32([0] * (rows + 1))
    kblk = torch.zeros(pages, 128, dtype=torch.bfloat16, device="cuda")
    lens = [130, 70, 0, 0]
    q, k, v = normal(1, 200, kv * group, 128, dt=torch.bfloat16), normal(2, 200, kv, 128, dt=torch.bfloat16), normal(3, 200, kv, 128, dt=torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    add.copy_(i32(lens)), cum.copy_(i32(cu(lens)))
    qsa.prompt_attention(q, k, v, cum, cum, out, lse, ws=aws)
    check_attention(out, lse, paged.prompt(q.double(), k.double(), v.double(), lens, lens, 128 ** -0.5), torch.bfloat16)
    qsa.pages_reserve(table, n, refs, add, new, cs, cd, ws=ws)
    qsa.pages_append(k, v, table, n, cum, kc, vc, ws=ws)
    n.copy_(new)
    side = [[k[:130], v[:130]], [k[130:], v[130:]], None, None]
    qsa.pages_fork(table, n, refs, i32([0, 1]), i32([2, 3]), ws=ws)
    side[2], side[3] = list(side[0]), list(side[1])

    nodes = [5, 3, 4, 6]
    total = sum(nodes)
    dq, dk, dv = (normal(7, total, h, 128, dt=torch.bfloat16) for h in (kv * group, kv, kv))
    parents, cun = i32([0] * total), i32(cu(nodes))
    tout, tlse = torch.empty_like(dq), torch.empty(dq.shape[:2], device="cuda")
    accepted = torch.full((total,), -1, dtype=torch.int32, device="cuda")

    def step():
        qsa.tree_attention(dq, dk, dv, parents, cun, 16, kc, vc, table, n, tout, tlse, ws=aws)
        qsa.pages_reserve(table, n, refs, add, new, cs, cd, ws=ws)
        qsa.pages_copy([kc.view(kv, pages, 64, 128), vc, kblk], cs, cd, ws=ws)
        qsa.pages_append(dk, dv, table, n, cum, kc, vc, rows=accepted, ws=ws)
        n.copy_(new)

    graph = None
    for turn in range(6):
        dq.copy_(normal(10 + turn, *dq.shape, dt=torch.bfloat16))
        dk.copy_(normal(20 + turn, *dk.shape, dt=torch.bfloat16)), dv.copy_(normal(30 + turn, *dv.shape, dt=torch.bfloat16))
        par = random_parents(turn, nodes)
        parents.copy_(i32(par))
        took, path = [], []
        for s, m in enumerate(nodes):                    # accept a path from some node up
            at, up = (turn + s) % m, []
            while at >= 0:
                up.append(at)
                at = par[cu(nodes)[s] + at]
            took.append(len(up)), path.extend(cu(nodes)[s] + x for x in reversed(up))
        add.copy_(i32(took)), cum.copy_(i32(cu(took)))
        accepted.fill_(-1)
        accepted[:len(path)] = i32(path)
        want = [paged.attended(dq[a:b].double(), torch.cat((side[s][0], dk[a:b])).double(), torch.cat((side[s][1], dv[a:b])).double(),
                               torch.cat((torch.ones(b - a, len(side[s][0]), dtype=torch.bool),
                                          torch.tensor(paged.ancestors(par[a:b]))), 1).cuda(), 128 ** -0.5)
                for s, (a, b) in enumerate(zip(cu(nodes), cu(nodes)[1:]))]
        if captured and graph is None:
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step()
        if captured:
            graph.replay()
        else:
            step()
        check_attention(tout, tlse, [torch.cat(x) for x in zip(*want)], torch.bfloat16)
        for s in range(rows):
            mine = path[sum(took[:s]):sum(took[:s + 1])]
            side[s] = [torch.cat((side[s][0], dk[mine])), torch.cat((side[s][1], dv[mine]))]
        assert n.tolist() == [len(x[0]) for x in side]
        if turn == 3:                                    # drop one, move the pages together
            keep = i32([-1, 0, -1, -1])
            qsa.pages_release(table, n, refs, keep, ws=ws)
            mv, to = (torch.empty(pages // 2, dtype=torch.int32, device="cuda") for _ in range(2))
            qsa.pages_compact(table, refs, table, refs, mv, to, ws=ws)
            qsa.pages_copy([kc.view(kv, pages, 64, 128), vc, kblk], mv, to, ws=ws)
            live = int((refs > 0).sum())
            assert (refs[:live] > 0).all() and (refs[live:] == 0).all()
            qsa.pages_fork(table, n, refs, i32([3]), i32([1]), ws=ws)
            side[1] = list(side[3])
        for s in range(rows):                            # the pages hold the rows
            pk, pv, ok = paged.paged_rows(kc, vc, table[s].tolist(), len(side[s][0]))
            assert ok.all() and torch.equal(pk, side[s][0]) and torch.equal(pv, side[s][1])
    held = table[table >= 0].long()
    assert torch.equal(torch.bincount(held, minlength=pages).int(), refs)
    assert qsa.read_flags(ws) == 0 and qsa.read_flags(aws) == 0
