"""The paged 16-bit cache and the dense attentions on the CPU: pins of their definition, and the argument
checks of the library and of the binding (no kernel runs)."""
import math

import pytest

torch = pytest.importorskip("torch")

from oracle import paged  # noqa: E402
from sparse_attention_kv_gb300 import _build, qsa  # noqa: E402

FAKE = 1 << 20
STEP = 1 << 34          # far enough apart that nothing overlaps


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return qsa.load()


# ------------------------------------------------------------------ the definition

def test_one_key_gives_its_value():
    q, k, v = torch.randn(1, 4, 128).double(), torch.randn(1, 2, 128).double(), torch.randn(1, 2, 128).double()
    out, lse, mass, _ = paged.prompt(q, k, v, [1], [1], 0.5)
    assert torch.equal(out[0], v[0].repeat_interleave(2, 0)) and torch.equal(mass, out.abs())
    assert torch.allclose(lse[0], 0.5 * (q[0] * k[0].repeat_interleave(2, 0)).sum(-1))


def test_equal_keys_give_means_and_no_key_gives_zero():
    q, v = torch.randn(4, 1, 128).double(), torch.randn(2, 1, 128).double()
    out, lse, _, _ = paged.prompt(q, torch.zeros(2, 1, 128).double(), v, [4], [2], 1.0)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()          # rows 0 and 1 see nothing
    assert torch.equal(out[2, 0], v[0, 0]) and lse[2, 0] == 0
    assert torch.allclose(out[3, 0], v[:, 0].mean(0)) and math.isclose(float(lse[3, 0]), math.log(2))


def test_causal_rows_are_the_prefixes():
    q, k, v = (torch.randn(7, 1, 128).double() for _ in "qkv")
    out, lse, _, _ = paged.prompt(q, k, v, [7], [7], 0.1)
    for i in range(7):
        z = 0.1 * (k[:i + 1, 0] @ q[i, 0])
        assert torch.allclose(out[i, 0], torch.softmax(z, 0) @ v[:i + 1, 0])
        assert torch.allclose(lse[i, 0], torch.logsumexp(z, 0))


def test_ancestors_by_hand():
    see = paged.ancestors([-1, 0, 0, 1, -1, 5, 2])      # node 5 names itself: as none
    want = [[0], [0, 1], [0, 2], [0, 1, 3], [4], [5], [0, 2, 6]]
    assert [[j for j, x in enumerate(r) if x] for r in see] == want


def test_a_chain_of_drafts_is_causal_attention():
    n, m, kv = 70, 5, 2
    kc, vc = torch.randn(kv, 3 * 64, 128).double(), torch.randn(kv, 3, 128, 64).double()
    q, k, v = torch.randn(m, 4, 128).double(), torch.randn(m, kv, 128).double(), torch.randn(m, kv, 128).double()
    pk, pv, ok = paged.paged_rows(kc, vc, [2, 0], n)
    assert ok.all() and torch.equal(pk[65], kc[:, 1]) and torch.equal(pv[3], vc[:, 2, :, 3])
    got = paged.tree(q, k, v, [-1, 0, 1, 2, 3], [m], kc, vc, [[2, 0]], [n], 0.1)
    want = paged.prompt(q, torch.cat((pk, k)), torch.cat((pv, v)), [m], [n + m], 0.1)
    for a, b in zip(got, want):
        assert torch.allclose(a, b)


def test_pages_by_hand():
    p = paged.Pool([[2, 0, -1], [-1] * 3, [-1] * 3], [100, 0, 0], [1, 0, 1, 0, 0])
    p.fork([0, 0], [1, 2])
    assert p.table == [[2, 0, -1]] * 3 and p.n == [100] * 3 and p.refs == [3, 0, 3, 0, 0]
    new, src, dst = p.reserve([1, 40, 0])               # rows 0 and 1 write page 0; row 2 keeps it
    assert new == [101, 140, 100] and src == [0, 0, -1] and dst == [1, 3, -1]
    assert p.table == [[2, 1, -1], [2, 3, 4], [2, 0, -1]] and p.refs == [1, 1, 3, 1, 1]
    p.release([0, -1, 64])
    assert p.table == [[-1] * 3, [2, 3, 4], [2, -1, -1]] and p.refs == [0, 0, 2, 1, 1] and p.n == [0, 100, 64]
    assert p.compact() == ([[-1] * 3, [2, 0, 1], [2, -1, -1]], [1, 1, 2, 0, 0], [3, 4], [0, 1])
    assert not p.flags


def test_fork_by_hand_from_a_row_with_entries_that_are_no_page():
    p = paged.Pool([[0, -1, 9, 1], [-1] * 4, [-1] * 4], [200, 0, 0], [1, 1, 0])
    p.fork([0], [1])
    assert p.table[1] == [0, -1, -1, 1] and p.n[1] == 200 and p.refs == [2, 2, 0] and p.flags == {"id"}
    p = paged.Pool([[0, 1], [-1] * 2, [-1] * 2], [300, 0, -7], [1, 1])
    p.fork([0], [1])
    assert p.table[1] == [0, 1] and p.n == [300, 128, -7] and p.refs == [2, 2] and p.flags == {"clamp"}


def test_reserve_by_hand_when_pages_run_out():
    p = paged.Pool([[0, -1], [1, -1], [2, -1]], [64, 64, 10], [1, 1, 1, 0])
    new, _, _ = p.reserve([1, 1, 1])                    # one free page: row 0 has it, row 2 needs none
    assert new == [65, 64, 11] and p.table == [[0, 3], [1, -1], [2, -1]] and p.flags == {"pages"}
    p = paged.Pool([[0], [1]], [64, 3], [1, 1])
    assert p.reserve([1, -2])[0] == [64, 3] and p.flags == {"clamp"}


def test_a_row_that_found_no_pages_appends_nothing():
    """A fork that goes on from within its parent's last page, in a full pool: without its end it writes there."""
    k = torch.arange(5.0)[:, None, None].expand(5, 1, 128).double() + 1
    for end in (False, True):
        p = paged.Pool([[0, 1, -1], [0, 1, -1]], [128, 100], [2, 2])
        new, src, dst = p.reserve([0, 5])
        assert new == [128, 100] and src == dst == [-1, -1] and p.flags == {"pages"} and p.table[1] == [0, 1, -1]
        kc, vc = torch.zeros(1, 128, 128).double(), torch.zeros(1, 2, 128, 64).double()
        p.append(k, k, p.n, [0, 0, 5], kc, vc, end=new if end else None)
        assert bool(kc.any()) == bool(vc.any()) == (not end)       # the other's tokens 100 .. 104


def test_reserve_by_hand_over_a_shared_page_behind_the_tokens():
    """Row 1's length was lowered by hand: page 1 behind its tokens is row 0's too.  Released, it gets a page of its own."""
    p = paged.Pool([[0, 1, -1], [0, 1, -1], [2, -1, -1]], [128, 64, 64], [2, 2, 1, 0, 0])
    assert p.reserve([0, 5, 1]) == ([128, 64, 65], [-1] * 3, [-1] * 3) and p.flags == {"id"}
    assert p.table == [[0, 1, -1], [0, 1, -1], [2, 3, -1]] and p.refs == [2, 2, 1, 1, 0]
    p.flags.clear()
    p.release([-1, 64, -1])
    assert p.reserve([0, 5, 0])[0] == [128, 69, 64] and p.table[1] == [0, 4, -1] and p.refs == [2, 1, 1, 1, 1] and not p.flags


def test_rows_behind_a_descent_take_no_entries():
    k = torch.arange(6.0)[:, None, None].expand(6, 1, 128).double() + 1
    p = paged.Pool([[0], [1], [2]], [0] * 3, [1] * 3)
    kc, vc = torch.zeros(1, 192, 128).double(), torch.zeros(1, 3, 128, 64).double()
    p.append(k, k, [0, 0, 0], [0, 6, 0, 6], kc, vc)
    assert torch.equal(kc[0, :6, 0], k[:, 0, 0]) and not kc[:, 6:].any() and p.flags == {"clamp"}


# ------------------------------------------------------------------ refusals of the library

STATUS = {"ARG": qsa.ERR_INVALID_ARG, "UNSUPPORTED": qsa.ERR_UNSUPPORTED, "WS": qsa.ERR_WORKSPACE, "OK": qsa.OK}
TABLE = [(dict(table=None), "ARG"), (dict(refs=None), "ARG"), (dict(rows=0), "ARG"), (dict(rows=4097), "ARG"),
         (dict(pages=0), "ARG"), (dict(pages=(1 << 20) + 1), "ARG"), (dict(width=0), "ARG"), (dict(width=(1 << 20) + 1, stride=1 << 21), "ARG"),
         (dict(stride=9), "ARG"), (dict(ws=FAKE + 64), "WS"), (dict(ws_bytes=128), "WS")]


def _args(names, **fixed):
    """Pointers far apart for the names, and the other arguments' values."""
    a = {n: FAKE + STEP * (i + 1) for i, n in enumerate(names)}
    a.update(rows=4, pages=100, width=10, stride=12, ws=FAKE, ws_bytes=1 << 20)
    a.update(fixed)
    return a


def _expect(lib, st, status):
    assert st == STATUS[status]
    assert status == "OK" or lib.qsa_last_error().decode()


@pytest.mark.parametrize("case,status", TABLE + [
    (dict(n=None), "ARG"), (dict(src=None), "ARG"), (dict(dst=None), "ARG"), (dict(count=-1), "ARG"), (dict(count=5), "ARG"),
    (dict(count=0), "OK"), (dict(src="n"), "ARG"), (dict(dst="table+180"), "ARG"), (dict(refs="n+12"), "ARG"),
    (dict(count=0, ws=None, ws_bytes=0), "OK")])
def test_fork_rejects_bad_arguments_before_launch(lib, case, status):
    a = _resolve(_args(["table", "n", "refs", "src", "dst"], count=3), case)
    _expect(lib, lib.qsa_pages_fork(a["table"], a["stride"], a["width"], a["n"], a["rows"], a["refs"], a["pages"], a["src"],
                                    a["dst"], a["count"], a["ws"], a["ws_bytes"], None), status)


def _resolve(a, case):
    """'name+bytes' in a case points into another array."""
    for k, v in case.items():
        if isinstance(v, str):
            name, _, off = v.partition("+")
            v = a[name] + int(off or 0)
        a[k] = v
    return a


def test_an_empty_array_overlaps_nothing(lib):
    """Of no entries, cut from an arena anywhere."""
    a = _args(["table", "n", "refs", "src", "dst", "k", "v", "cu", "first", "kc", "vc", "idx"])
    t = (a["table"], a["stride"], a["width"])
    for at in (a["table"] + 40, a["n"] + 4, a["refs"] + 8):
        _expect(lib, lib.qsa_pages_fork(*t, a["n"], 4, a["refs"], 100, at, at, 0, None, 0, None), "OK")
    packed = (qsa.BlockArray * 1)(qsa.BlockArray(a["kc"], a["kc"], 64, 1, 8, 8))
    _expect(lib, lib.qsa_pages_copy(packed, 1, a["kc"] + 64, a["kc"] + 64, 0, None, 0, None), "OK")
    for k, idx in ((a["kc"] + 256, a["idx"]), (a["k"], a["vc"] + 256)):
        _expect(lib, lib.qsa_pages_append(k, 512, 128, a["v"], 512, 128, qsa.BF16, 0, idx, 0, a["cu"], a["first"], *t, 4, 4, 128, a["kc"],
                                          a["vc"], 6400, None, 0, None), "OK")


@pytest.mark.parametrize("case,status", TABLE + [
    (dict(n=None), "ARG"), (dict(keep=None), "ARG"), (dict(keep="n+4"), "ARG"), (dict(keep="refs"), "ARG"), (dict(n="table"), "ARG")])
def test_release_rejects_bad_arguments_before_launch(lib, case, status):
    a = _resolve(_args(["table", "n", "refs", "keep"]), case)
    _expect(lib, lib.qsa_pages_release(a["table"], a["stride"], a["width"], a["n"], a["rows"], a["refs"], a["pages"], a["keep"],
                                       a["ws"], a["ws_bytes"], None), status)


@pytest.mark.parametrize("case,status", TABLE + [
    (dict(n=None), "ARG"), (dict(add=None), "ARG"), (dict(new=None), "ARG"), (dict(src=None), "ARG"), (dict(dst=None), "ARG"),
    (dict(ws=None), "WS"), (dict(ws_bytes=256), "WS"), (dict(new="n"), "ARG"), (dict(new="add+12"), "ARG"), (dict(dst="src+8"), "ARG"),
    (dict(src="table"), "ARG"), (dict(refs="add"), "ARG")])
def test_reserve_rejects_bad_arguments_before_launch(lib, case, status):
    a = _resolve(_args(["table", "n", "refs", "add", "new", "src", "dst"]), case)
    _expect(lib, lib.qsa_pages_reserve(a["table"], a["stride"], a["width"], a["n"], a["rows"], a["refs"], a["pages"], a["add"],
                                       a["new"], a["src"], a["dst"], a["ws"], a["ws_bytes"], None), status)


@pytest.mark.parametrize("case,status", TABLE + [
    (dict(tout=None), "ARG"), (dict(rout=None), "ARG"), (dict(src=None), "ARG"), (dict(dst=None), "ARG"), (dict(ws=None), "WS"),
    (dict(ws_bytes=256), "WS"), (dict(tout="table+4"), "ARG"), (dict(rout="refs+4"), "ARG"), (dict(src="dst+100"), "ARG"),
    (dict(dst="rout"), "ARG"), (dict(src="table"), "ARG")])
def test_compact_rejects_bad_arguments_before_launch(lib, case, status):
    a = _resolve(_args(["table", "refs", "tout", "rout", "src", "dst"]), case)
    _expect(lib, lib.qsa_pages_compact(a["table"], a["stride"], a["width"], a["rows"], a["refs"], a["pages"], a["tout"], a["rout"],
                                       a["src"], a["dst"], a["ws"], a["ws_bytes"], None), status)


@pytest.mark.parametrize("arrays,n,status", [
    ([], 4, "ARG"), ([(FAKE, FAKE, 64, 1, 8, 8)] * 9, 4, "ARG"), ([(FAKE, STEP, 64, 1, 8, 8)], 4, "ARG"),
    ([(None, None, 64, 1, 8, 8)], 4, "ARG"), ([(FAKE, FAKE, 64, 0, 8, 8)], 4, "ARG"), ([(FAKE, FAKE, 64, 1, 8, 9)], 4, "ARG"),
    ([(FAKE, FAKE, 64, 1, 0, 0)], 4, "ARG"), ([(FAKE, FAKE, 6, 1, 8, 8)], 4, "ARG"), ([(FAKE + 2, FAKE + 2, 64, 1, 8, 8)], 4, "ARG"),
    ([(FAKE, FAKE, 64, 1, 8, 8), (FAKE + 448, FAKE + 448, 64, 1, 8, 8)], 4, "ARG"), ([(FAKE, FAKE, 64, 1, 8, 8)], -1, "ARG"),
    ([(FAKE, FAKE, 64, 1, 8, 8)], (1 << 20) + 1, "ARG"), ([(2 * STEP - 256, 2 * STEP - 256, 64, 1, 8, 8)], 4, "ARG"),
    ([(FAKE, FAKE, 64, 1, 8, 8)], 0, "OK")])
def test_copy_rejects_bad_arguments_before_launch(lib, arrays, n, status):
    packed = (qsa.BlockArray * max(1, len(arrays)))(*(qsa.BlockArray(*x) for x in arrays))
    _expect(lib, lib.qsa_pages_copy(packed, len(arrays), 2 * STEP, 3 * STEP, n, None, 0, None), status)


@pytest.mark.parametrize("case,status", [
    (dict(k=None), "ARG"), (dict(v=None), "ARG"), (dict(cu=None), "ARG"), (dict(first=None), "ARG"), (dict(table=None), "ARG"),
    (dict(kc=None), "ARG"), (dict(vc=None), "ARG"), (dict(k=FAKE + 8), "ARG"), (dict(kc=FAKE + 8), "ARG"), (dict(ks=(12, 128)), "ARG"),
    (dict(vs=(512, 4)), "ARG"), (dict(ks=(-512, 128)), "ARG"), (dict(D=64), "ARG"), (dict(kv=0), "ARG"), (dict(kv=65536), "ARG"),
    (dict(cap=100), "ARG"), (dict(cap=0), "ARG"), (dict(rows=0), "ARG"), (dict(rows=4097), "ARG"), (dict(stride=9), "ARG"),
    (dict(n=-1), "ARG"), (dict(n=(1 << 28) + 1), "ARG"), (dict(source=-1), "ARG"), (dict(idx=None, n=5), "ARG"), (dict(kc="k"), "ARG"),
    (dict(vc="kc+65536"), "ARG"), (dict(kc="table"), "ARG"), (dict(dt=qsa.F32), "UNSUPPORTED"), (dict(dt=qsa.E4M3), "UNSUPPORTED"),
    (dict(ws=FAKE + 8), "WS"), (dict(ws_bytes=255), "WS"), (dict(n=0), "OK"), (dict(n=0, ws=None, ws_bytes=0), "OK")])
def test_append_rejects_bad_arguments_before_launch(lib, case, status):
    a = _resolve(_args(["k", "v", "idx", "cu", "first", "table", "kc", "vc"], ks=(512, 128), vs=(512, 128), dt=qsa.BF16, source=8, n=4,
                       kv=4, D=128, cap=6400), case)
    _expect(lib, lib.qsa_pages_append(a["k"], *a["ks"], a["v"], *a["vs"], a["dt"], a["source"], a["idx"], a["n"], a["cu"], a["first"],
                                      a["table"], a["stride"], a["width"], a["rows"], a["kv"], a["D"], a["kc"], a["vc"], a["cap"],
                                      a["ws"], a["ws_bytes"], None), status)


@pytest.mark.parametrize("case,status", [
    (dict(end=None), "ARG"), (dict(end="kc+64"), "ARG"), (dict(vc="end"), "ARG"), (dict(k=None), "ARG"), (dict(first=None), "ARG"),
    (dict(kc=FAKE + 8), "ARG"), (dict(ks=(12, 128)), "ARG"), (dict(D=64), "ARG"), (dict(cap=100), "ARG"), (dict(rows=4097), "ARG"),
    (dict(n=-1), "ARG"), (dict(idx=None, n=5), "ARG"), (dict(dt=qsa.F32), "UNSUPPORTED"), (dict(ws_bytes=255), "WS"), (dict(n=0), "OK"),
    (dict(n=0, end="first"), "OK")])
def test_append_reserved_rejects_bad_arguments_before_launch(lib, case, status):
    a = _resolve(_args(["k", "v", "idx", "cu", "first", "end", "table", "kc", "vc"], ks=(512, 128), vs=(512, 128), dt=qsa.BF16, source=8,
                       n=4, kv=4, D=128, cap=6400), case)
    _expect(lib, lib.qsa_pages_append_reserved(a["k"], *a["ks"], a["v"], *a["vs"], a["dt"], a["source"], a["idx"], a["n"], a["cu"],
                                               a["first"], a["end"], a["table"], a["stride"], a["width"], a["rows"], a["kv"], a["D"],
                                               a["kc"], a["vc"], a["cap"], a["ws"], a["ws_bytes"], None), status)


@pytest.mark.parametrize("name,over,status", [
    (c, o, "ARG") for c, os in dict(fork="table+0 n+0 refs+0 src+0 dst+0", release="table+0 n+0 refs+0 keep+0",
                                    reserve="table+0 n+0 refs+0 add+0 new+0 src+0 dst+0", compact="table+0 refs+0 tout+0 rout+0 src+0 dst+0",
                                    append="k+0 v+0 idx+0 cu+0 first+0 table+0 kc+256 vc+1638144",
                                    append_reserved="k+0 end+0 kc+1638144", copy="pool+0 pool+8448 ids+0 to+0").items() for o in os.split()] + [
    # the workspace begins before the array and reaches into it; and right in front of it and behind it
    ("fork", "table-256", "OK"), ("fork", "table-0", "ARG"), ("reserve", "refs-512", "ARG"), ("reserve", "refs-256", "ARG"),
    ("compact", "rout-512", "ARG"), ("copy", "pool-256", "OK"), ("copy", "pool+12800", "OK"), ("append", "kc-256", "OK")])
def test_a_workspace_that_overlaps_is_refused(lib, name, over, status):
    """100 pages, 4 rows: fork, release, copy and append use 256 bytes of it, reserve and compact 768."""
    names = ["table", "n", "refs", "src", "dst", "keep", "add", "new", "tout", "rout", "k", "v", "idx", "cu", "first", "end", "kc", "vc",
             "pool", "ids", "to"]
    a = _args(names, ks=(512, 128), vs=(512, 128))
    for n in names:
        a[n] &= ~255
    array, sign, off = over.partition("+" if "+" in over else "-")
    ws = (a[array] + int(sign + off), 4096)
    t, tail = (a["table"], a["stride"], a["width"]), (*ws, None)
    assert lib.qsa_pages_workspace_bytes(4, 100) == 768
    if name == "fork":          # of no rows: a call that passes the checks launches nothing
        count = 0 if status == "OK" else 3
        st = lib.qsa_pages_fork(*t, a["n"], 4, a["refs"], 100, a["src"], a["dst"], count, *tail)
    elif name == "release":
        st = lib.qsa_pages_release(*t, a["n"], 4, a["refs"], 100, a["keep"], *tail)
    elif name == "reserve":
        st = lib.qsa_pages_reserve(*t, a["n"], 4, a["refs"], 100, a["add"], a["new"], a["src"], a["dst"], *tail)
    elif name == "compact":
        st = lib.qsa_pages_compact(*t, 4, a["refs"], 100, a["tout"], a["rout"], a["src"], a["dst"], *tail)
    elif name == "copy":
        packed = (qsa.BlockArray * 1)(qsa.BlockArray(a["pool"], a["pool"], 128, 1, 100, 100))
        st = lib.qsa_pages_copy(packed, 1, a["ids"], a["to"], 0 if status == "OK" else 4, *tail)
    else:
        n = 0 if status == "OK" else 4
        end = (a["end"],) if name == "append_reserved" else ()
        f = getattr(lib, "qsa_pages_" + name)
        st = f(a["k"], 512, 128, a["v"], 512, 128, qsa.BF16, 8, a["idx"], n, a["cu"], a["first"], *end, *t, 4, 1, 128, a["kc"], a["vc"],
               6400, *tail)
    _expect(lib, st, status)


DENSE = [
    (dict(q=None), "ARG"), (dict(k=None), "ARG"), (dict(v=None), "ARG"), (dict(cu=None), "ARG"), (dict(out=None), "ARG"),
    (dict(q=FAKE + 8), "ARG"), (dict(v=FAKE + 2), "ARG"), (dict(out=FAKE + 8), "ARG"), (dict(qs=(100, 128)), "ARG"),
    (dict(qs=(8192, -128)), "ARG"), (dict(ks=(64, 128)), "ARG"), (dict(vs=(512, 0)), "ARG"), (dict(D=64), "ARG"), (dict(kv=0), "ARG"),
    (dict(heads=0), "ARG"), (dict(heads=63), "ARG"), (dict(heads=68), "ARG"), (dict(seqs=0), "ARG"), (dict(seqs=65536), "ARG"),
    (dict(total=-1), "ARG"), (dict(total=1 << 25), "ARG"), (dict(scale=0.0), "ARG"), (dict(scale=float("nan")), "ARG"),
    (dict(scale=float("inf")), "ARG"), (dict(odt=qsa.F16), "ARG"), (dict(out="q"), "ARG"), (dict(lse="k+256"), "ARG"),
    (dict(lse="out"), "ARG"), (dict(ws="v"), "ARG"), (dict(dt=qsa.F32), "UNSUPPORTED"), (dict(dt=qsa.E4M3), "UNSUPPORTED"),
    (dict(ws=None), "WS"), (dict(ws=FAKE + 64), "WS"), (dict(ws_bytes=4096), "WS"), (dict(total=0), "OK")]


def _dense(case, names, **fixed):
    return _resolve(_args(["q", "k", "v", "cu", "out", "lse", *names], qs=(8192, 128), ks=(512, 128), vs=(512, 128), dt=qsa.BF16, seqs=4,
                          total=20, heads=64, kv=4, D=128, scale=0.1, odt=qsa.BF16, ws_bytes=1 << 28, **fixed), case)


@pytest.mark.parametrize("case,status", DENSE + [(dict(cuk=None), "ARG"), (dict(keys=-1), "ARG"), (dict(keys=1 << 30), "ARG"),
                                                 (dict(out="cuk"), "ARG")])
def test_prompt_attention_rejects_bad_arguments_before_launch(lib, case, status):
    a = _dense(case, ["cuk"], keys=30)
    _expect(lib, lib.qsa_prompt_attention(a["q"], *a["qs"], a["k"], *a["ks"], a["v"], *a["vs"], a["dt"], a["cu"], a["cuk"], a["seqs"],
                                          a["total"], a["keys"], a["heads"], a["kv"], a["D"], a["scale"], a["out"], a["odt"],
                                          a["lse"], a["ws"], a["ws_bytes"], None), status)


@pytest.mark.parametrize("case,status", DENSE + [
    (dict(parents=None), "ARG"), (dict(kc=None), "ARG"), (dict(vc=None), "ARG"), (dict(table=None), "ARG"), (dict(n=None), "ARG"),
    (dict(most=0), "ARG"), (dict(most=65), "ARG"), (dict(cap=100), "ARG"), (dict(cap=0), "ARG"), (dict(cap=64 * ((1 << 20) + 1)), "ARG"),
    (dict(cap=1 << 26, kv=16, heads=64), "ARG"), (dict(width=0), "ARG"), (dict(stride=9), "ARG"), (dict(kc=FAKE + 8), "ARG"),
    (dict(out="kc"), "ARG"), (dict(lse="table"), "ARG"), (dict(out="parents"), "ARG")])
def test_tree_attention_rejects_bad_arguments_before_launch(lib, case, status):
    a = _dense(case, ["parents", "kc", "vc", "table", "n"], most=16, cap=6400)
    _expect(lib, lib.qsa_tree_attention(a["q"], *a["qs"], a["k"], *a["ks"], a["v"], *a["vs"], a["dt"], a["parents"], a["cu"], a["seqs"],
                                        a["total"], a["most"], a["kc"], a["vc"], a["cap"], a["table"], a["stride"], a["width"],
                                        a["n"], a["heads"], a["kv"], a["D"], a["scale"], a["out"], a["odt"], a["lse"], a["ws"],
                                        a["ws_bytes"], None), status)


def test_workspace_sizes(lib):
    assert lib.qsa_pages_workspace_bytes(64, 4096) >= 256 + 4 * (64 + 4096 + 1) and lib.qsa_pages_workspace_bytes(64, 4096) % 256 == 0
    for bad in ((0, 1), (4097, 1), (1, 0), (1, (1 << 20) + 1)):
        assert lib.qsa_pages_workspace_bytes(*bad) == 0
    one, many = lib.qsa_attention_workspace_bytes(1, 64, 4), lib.qsa_attention_workspace_bytes(100_000, 64, 4)
    assert 256 < one < many == lib.qsa_attention_workspace_bytes(9, 64, 4)      # 9 tokens of 16 heads begin a second stream
    for bad in ((0, 64, 4), (1, 63, 4), (1, 68, 4), (1, 0, 1), (1, 4, 0), (1 << 25, 64, 4)):
        assert lib.qsa_attention_workspace_bytes(*bad) == 0
    # never less for more rows
    sizes = [lib.qsa_attention_workspace_bytes(n, 7, 1) for n in range(1, 60)]
    assert sizes == sorted(sizes)


# ------------------------------------------------------------------ refusals of the binding

def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_binding_checks_the_pages(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)      # CPU tensors pass for the device's
    table, n, refs, two = _i32(4, 10), _i32(4), _i32(100), _i32(2)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    for bad in (dict(table=table.long()), dict(table=table[0]), dict(table=table.t()), dict(n_tokens=_i32(3)), dict(n_tokens=n.long()),
                dict(refs=refs[::2]), dict(src=_i32(3)), dict(dst=two.float())):
        a = dict(table=table, n_tokens=n, refs=refs, src=two, dst=two)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.pages_fork(**a)
    for bad in (dict(keep=two), dict(n_tokens=_i32(4, 1)), dict(refs=refs.short())):
        a = dict(table=table, n_tokens=n, refs=refs, keep=n)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.pages_release(**a)
    for bad in (dict(add=two), dict(new_tokens=n.float()), dict(copy_src=_i32(5)), dict(copy_dst=_i32(8)[::2])):
        a = dict(table=table, n_tokens=n, refs=refs, add=n, new_tokens=n, copy_src=n, copy_dst=n, ws=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.pages_reserve(**a)
    half = _i32(50)
    for bad in (dict(table_out=_i32(4, 11)), dict(table_out=_i32(4, 20)[:, :10]), dict(refs_out=half), dict(copy_src=refs), dict(copy_dst=_i32(49))):
        a = dict(table=table, refs=refs, table_out=table, refs_out=refs, copy_src=half, copy_dst=half, ws=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.pages_compact(**a)
    pool = torch.zeros(2, 8, 4)
    for arrays, src, dst in (([], two, two), ([pool] * 9, two, two), ([pool.transpose(0, 1)], two, two), ([pool], two, n), ([pool], two.long(), two)):
        with pytest.raises(ValueError):
            qsa.pages_copy(arrays, src, dst)
    rows, kc, vc = torch.zeros(6, 2, 128).half(), torch.zeros(2, 640, 128).half(), torch.zeros(2, 10, 128, 64).half()
    for bad in (dict(k=rows.float()), dict(v=rows.bfloat16()), dict(v=rows[:5]), dict(k=rows[:, :1], v=rows[:, :1]), dict(first=two),
                dict(cu_rows=n), dict(kcache=kc[:, :639]), dict(kcache=kc.bfloat16()), dict(vcache_t=vc[:, :9]), dict(rows=two.long()),
                dict(vcache_t=vc.transpose(2, 3))):
        a = dict(k=rows, v=rows, table=table, first=n, cu_rows=_i32(5), kcache=kc, vcache_t=vc)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.pages_append(**a)
    with pytest.raises(ValueError):
        qsa.alloc_pages(1, 1, 0, 1)
    with pytest.raises(ValueError):
        qsa.alloc_pages(1, 1, 4, 1, dtype=torch.float32)
    with pytest.raises(ValueError):
        qsa.alloc_pages_workspace(5000, 10)


@pytest.mark.parametrize("end", [_i32(3), _i32(4, 1), _i32(8)[::2], _i32(4).long()])
def test_binding_checks_where_an_append_ends(lib, monkeypatch, end):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    rows, kc, vc = torch.zeros(6, 2, 128).half(), torch.zeros(2, 640, 128).half(), torch.zeros(2, 10, 128, 64).half()
    with pytest.raises(ValueError, match="end"):
        qsa.pages_append(rows, rows, _i32(4, 10), _i32(4), _i32(5), kc, vc, end=end)


def test_binding_checks_the_attentions(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    q, k = torch.zeros(6, 8, 128).bfloat16(), torch.zeros(6, 2, 128).bfloat16()
    cu, ws = _i32(3), torch.zeros(1 << 16, dtype=torch.uint8)
    common = [dict(q=q.float()), dict(k=k.half()), dict(v=k[:5]), dict(q=q[..., ::2]), dict(out=q.half()), dict(out=q[:5]),
              dict(out=torch.zeros(6, 128, 8).bfloat16().transpose(1, 2)), dict(lse=torch.zeros(6, 7)), dict(lse=torch.zeros(6, 8).double())]
    for bad in common + [dict(cu_q=cu.long()), dict(cu_k=_i32(4))]:
        a = dict(q=q, k=k, v=k, cu_q=cu, cu_k=cu, out=torch.zeros_like(q), ws=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.prompt_attention(**a)
    kc, vc = torch.zeros(2, 640, 128).bfloat16(), torch.zeros(2, 10, 128, 64).bfloat16()
    for bad in common + [dict(k=k[:5], v=k[:5]), dict(parents=_i32(5)), dict(cu_nodes=_i32(4)), dict(n_tokens=_i32(3)), dict(table=_i32(2)),
                         dict(kcache=kc[:1], vcache_t=vc[:1]), dict(kcache=kc.half()), dict(vcache_t=vc[:, :9])]:
        a = dict(q=q, k=k, v=k, parents=_i32(6), cu_nodes=cu, max_nodes=4, kcache=kc, vcache_t=vc, table=_i32(2, 7), n_tokens=_i32(2),
                 out=torch.zeros_like(q), ws=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.tree_attention(**a)
    with pytest.raises(ValueError):
        qsa.alloc_attention_workspace(0, 8, 2)


def test_binding_refuses_other_devices(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    n = _i32(4)
    with pytest.raises(ValueError, match="current device"):
        qsa.pages_release(_i32(4, 10), n, _i32(100), n)
    q, k, cu = torch.zeros(6, 8, 128).half(), torch.zeros(6, 2, 128).half(), _i32(3)
    with pytest.raises(ValueError, match="current device"):
        qsa.prompt_attention(q, k, k, cu, cu, torch.zeros_like(q), ws=torch.zeros(256, dtype=torch.uint8))
