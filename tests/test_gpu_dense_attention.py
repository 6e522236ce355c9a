"""Prompt attention and tree attention on the GPU against their definition in 64 bits."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from oracle import paged  # noqa: E402
from sparse_attention_kv_gb300 import qsa  # noqa: E402

from .paged_cases import HALF, check_attention, cu, i32, normal, random_parents, random_pool, random_table  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16
SCALE = 128 ** -0.5


def _prompt(q, k, v, lq, lk, out_dt=None, lse=True, scale=None, ws=None, cu_q=None, cu_k=None):
    out = torch.full(q.shape, float("nan"), dtype=out_dt or q.dtype, device="cuda")
    ls = torch.full(q.shape[:2], float("nan"), device="cuda") if lse else None
    ws = qsa.alloc_attention_workspace(max(1, q.shape[0]), q.shape[1], k.shape[1]) if ws is None else ws
    qsa.prompt_attention(q, k, v, i32(cu(lq)) if cu_q is None else cu_q, i32(cu(lk)) if cu_k is None else cu_k, out, ls, ws=ws,
                         scale=scale)
    return out, ls, ws


def _check_prompt(lq, lk, kv, group, dt, seed=1, **kw):
    q, k, v = (normal(seed + i, n, h, 128, dt=dt, mean=m) for i, (n, h, m) in
               enumerate(((sum(lq), kv * group, 0.0), (sum(lk), kv, 0.0), (sum(lk), kv, 0.25))))
    out, lse, ws = _prompt(q, k, v, lq, lk, **kw)
    want = paged.prompt(q.double(), k.double(), v.double(), lq, lk, kw.get("scale") or SCALE)
    check_attention(out, lse, want, dt)
    assert qsa.read_flags(ws) == 0


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("kv,group", [(4, 16), (2, 7), (1, 1), (3, 2), (1, 16)])
@pytest.mark.parametrize("lq,lk", [([1], [1]), ([5], [5]), ([64], [64]), ([65, 1, 130], [65, 1, 130]), ([300, 17], [300, 17]),
                                   ([3], [500]), ([128, 129], [1000, 129])])
def test_prompt_matches_the_definition(lq, lk, kv, group, dt):
    _check_prompt(lq, lk, kv, group, dt)


@pytest.mark.parametrize("lq,lk", [([1021, 333, 1, 777], [1021, 850, 2001, 840]), ([2500], [2500]), ([16, 4000], [16, 4000]),
                                   ([1] * 40, list(range(1, 400, 10))), ([7], [9001])])
@pytest.mark.parametrize("kv,group,dt", [(2, 7, F16), (1, 16, BF16), (2, 1, BF16)])
def test_prompt_longer_and_ragged(lq, lk, kv, group, dt):
    _check_prompt(lq, lk, kv, group, dt, seed=11)


def test_prompt_rows_without_keys_are_zero():
    """More queries than keys, and no keys at all: the first rows see nothing."""
    lq, lk = [200, 3, 5, 1], [70, 3, 0, 1]
    _check_prompt(lq, lk, 2, 4, BF16, seed=3)
    q, k, v = normal(1, 4, 8, 128, dt=F16), *(torch.empty(0, 2, 128, dtype=F16, device="cuda") for _ in "kv")
    out, lse, ws = _prompt(q, k, v, [4], [0])
    assert (out == 0).all() and torch.isneginf(lse).all() and qsa.read_flags(ws) == 0


def test_prompt_fp32_output_no_lse_and_scale():
    _check_prompt([130, 9], [140, 9], 2, 3, F16, out_dt=torch.float32)
    _check_prompt([130, 9], [140, 9], 2, 3, BF16, out_dt=torch.float32, lse=False, scale=0.3)
    _check_prompt([130, 9], [140, 9], 2, 3, BF16, scale=2.0)


def test_prompt_strided_inputs():
    """Slices of a fused projection, head-major tensors, a broadcast query row."""
    row = normal(5, 150, 20 + 2 * 4, 128, dt=BF16)
    q, k, v = row[:, :20], row[:, 20:24], row[:, 24:]
    want = paged.prompt(q.double(), k.double(), v.double(), [100, 50], [100, 50], SCALE)
    out, lse, _ = _prompt(q, k, v, [100, 50], [100, 50])
    check_attention(out, lse, want, BF16)
    qh, kh, vh = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))   # head-major
    again, lse2, _ = _prompt(qh, kh, vh, [100, 50], [100, 50])
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    one = q[:1].expand(150, -1, -1)
    out, lse, _ = _prompt(one, k, v, [100, 50], [100, 50])
    want = paged.prompt(one.double(), k.double(), v.double(), [100, 50], [100, 50], SCALE)
    check_attention(out, lse, want, BF16)


@pytest.mark.parametrize("group", [1, 7, 16])
def test_prompt_unseen_rows_do_not_touch_it(group):
    """NaN and infinities in keys and values that no query, or only later queries, see."""
    lq, lk, kv = [70, 130], [70, 300], 2
    q, k, v = normal(1, 210, kv * group, 128, dt=BF16), normal(2, 380, kv, 128, dt=BF16), normal(3, 380, kv, 128, dt=BF16)
    good, lse, _ = _prompt(q, k, v, lq, lk)
    cq, ck = [5, 75, 205], [5, 75, 375]          # rows before the first and behind the last sequence
    qq = torch.cat((normal(4, 5, kv * group, 128, dt=BF16), q[:200], normal(5, 5, kv * group, 128, dt=BF16)))
    kk, vv = (torch.full((380, kv, 128), float("nan"), dtype=BF16, device="cuda") for _ in "kv")
    kk[5:375], vv[5:375] = k[:370], v[:370]
    vv[375:] = float("inf")
    out, ls, ws = _prompt(qq, kk, vv, None, None, cu_q=i32(cq), cu_k=i32(ck))
    assert torch.equal(out[5:205], good[:200]) and torch.equal(ls[5:205], lse[:200])
    assert torch.isnan(out[:5]).all() and torch.isnan(out[205:]).all() and torch.isnan(ls[:5]).all()   # left as they were
    assert qsa.read_flags(ws) == 0
    # keys of the second sequence's last tokens: only the queries at and behind them change
    for bad in (float("nan"), float("inf"), -float("inf")):
        k2, v2 = k.clone(), v.clone()
        k2[70 + 290] = bad
        v2[70 + 280, :, 5] = bad                 # seen by queries 110 ..
        out, ls, _ = _prompt(q, k2, v2, lq, lk)
        assert torch.equal(out[:70 + 110], good[:70 + 110]) and torch.equal(ls[:70 + 110], lse[:70 + 110])
        mid = out[70 + 110:70 + 120]             # the value's dimension, and no other
        assert not torch.isfinite(mid[..., 5]).any()
        if not math.isnan(bad):
            assert (mid[..., 5] == bad).all()
        keep = [d for d in range(128) if d != 5]
        assert torch.equal(mid[..., keep], good[70 + 110:70 + 120][..., keep])
        if math.isnan(bad):
            assert torch.isnan(out[70 + 120:]).all() and torch.isnan(ls[70 + 120:]).all()


@pytest.mark.parametrize("kv,group", [(1, 16), (2, 8), (3, 1), (1, 4), (2, 2)])
def test_prompt_writes_no_row_beyond_its_sequences(kv, group):
    """Sequences that end within a tile, a warp's rows, or with them; rows between and behind them stay as they were."""
    toks = 128 // group
    lens, gaps = [toks, 2 * toks, toks // 4, toks + 3 * toks // 4, 2 * toks + 1, 3], [0, 5, 1, 2, 7, 1, 9]
    total = sum(lens) + sum(gaps)
    q, k, v = normal(1, total, kv * group, 128, dt=F16), *(normal(2 + i, sum(lens), kv, 128, dt=F16) for i in range(2))
    full, fl, _ = _prompt(q[:sum(lens)], k, v, lens, lens)
    # the same sequences behind empty ones that own the gaps (no keys: rows of zeros), and with the gaps in no sequence
    at = a = 0
    qq = torch.empty_like(q)
    cq, ck, mine = [0], [0], torch.zeros(total, dtype=torch.bool)
    for gap, m in zip(gaps, lens):
        cq.append(at + gap), ck.append(ck[-1])
        at += gap
        qq[at:at + m] = q[a:a + m]
        mine[at:at + m] = True
        cq.append(at + m), ck.append(ck[-1] + m)
        at, a = at + m, a + m
    out, ls, ws = _prompt(qq, k, v, None, None, cu_q=i32(cq), cu_k=i32(ck))
    assert torch.equal(out[mine], full) and torch.equal(ls[mine], fl)
    inside = ~mine
    inside[at:] = False
    assert (out[inside] == 0).all() and torch.isnan(out[at:]).all() and torch.isnan(ls[at:]).all()
    assert qsa.read_flags(ws) == 0
    for n, m in ((0, lens[0]), (sum(lens[:2]), lens[2])):         # one sequence in a larger output
        out, ls, _ = _prompt(q, k, v, None, None, cu_q=i32([n, n + m]), cu_k=i32([n, n + m]))
        check_attention(out[n:n + m], ls[n:n + m], paged.prompt(q[n:n + m].double(), k[n:n + m].double(), v[n:n + m].double(), [m], [m], SCALE), F16)
        assert torch.isnan(out[:n]).all() and torch.isnan(out[n + m:]).all()


def test_prompt_bad_ranges_are_flagged():
    q, k, v = normal(1, 40, 4, 128, dt=BF16), normal(2, 40, 2, 128, dt=BF16), normal(3, 40, 2, 128, dt=BF16)
    good, lse, _ = _prompt(q, k, v, [40], [40])
    out, ls, ws = _prompt(q, k, v, None, None, cu_q=i32([0, 99]), cu_k=i32([-3, 40]))
    assert torch.equal(out, good) and qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED
    out, ls, ws = _prompt(q, k, v, None, None, cu_q=i32([0, 40, 7]), cu_k=i32([0, 40, 40]))
    assert torch.equal(out, good) and qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED


def test_sequences_that_overlap_are_refused_on_the_device():
    q, k, v = normal(1, 40, 4, 128, dt=BF16), normal(2, 40, 2, 128, dt=BF16), normal(3, 40, 2, 128, dt=BF16)
    out, ls, ws = _prompt(q, k, v, None, None, cu_q=i32([0, 30, 5, 40]), cu_k=i32([0, 10, 20, 40]))
    assert torch.isnan(out).all() and torch.isnan(ls).all() and qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED
    good, lse, _ = _prompt(q, k, v, [40], [40])          # keys may be shared: both sequences see the first 20
    out, ls, ws = _prompt(q, k, v, [20, 20], None, cu_k=i32([0, 20, 0]))
    assert torch.equal(out[:20], good[:20]) and (out[20:] == 0).all() and qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED


def test_prompt_large_logits_and_late_rises():
    """Logits in the hundreds, and a maximum that rises in every tile."""
    for dt in (BF16, F16):
        q, k, v = normal(1, 600, 4, 128, dt=dt), normal(2, 600, 2, 128, dt=dt), normal(3, 600, 2, 128, dt=dt)
        rise = torch.linspace(0.1, 6.0, 600, device="cuda")[:, None, None]
        k2 = (k.float() * rise).to(dt)
        out, lse, _ = _prompt(q, k2, v, [600], [600])
        check_attention(out, lse, paged.prompt(q.double(), k2.double(), v.double(), [600], [600], SCALE), dt)
        k2[:, :, :] = (q[:, :1] * rise).to(dt)      # aligned keys: each later key dominates by far
        out, lse, _ = _prompt(q, k2, v, [600], [600])
        check_attention(out, lse, paged.prompt(q.double(), k2.double(), v.double(), [600], [600], SCALE), dt)


def test_prompt_is_the_same_every_time_and_in_any_batch():
    q, k, v = normal(1, 900, 8, 128, dt=BF16), normal(2, 900, 2, 128, dt=BF16), normal(3, 900, 2, 128, dt=BF16)
    ws = qsa.alloc_attention_workspace(900, 8, 2)
    first, l1, _ = _prompt(q, k, v, [500, 400], [500, 400], ws=ws)
    for _ in range(3):
        out, ls, _ = _prompt(q, k, v, [500, 400], [500, 400], ws=ws)
        assert torch.equal(out, first) and torch.equal(ls, l1)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("lq,lk", [([300], [300]), ([3], [5000]), ([40, 900], [700, 900])])
def test_a_constant_value_comes_back_within_a_weights_rounding(lq, lk, dt):
    """The weights of the product are rounded, those that are summed are not: each term is off by HALF[dt] of itself at most, so the
    sum is; 2^-14 for fp32 sums, and half fp16's least step, 2^-25, for each weight below its normal range, the largest being 1 at
    least, as in check_attention.  Late keys that outweigh the others by up to 2^8 are the worst case for it."""
    q, k = normal(1, sum(lq), 16, 128, dt=dt), normal(2, sum(lk), 1, 128, dt=dt)
    k[1::7] = (q[:1, :1] * torch.linspace(0.0, 0.4, k[1::7].shape[0], device="cuda")[:, None, None]).to(dt)
    v = torch.full_like(k, 1.3)
    out, lse, _ = _prompt(q, k, v, lq, lk, out_dt=torch.float32)
    assert ((out.double() / v[0, 0, 0].double() - 1).abs() <= HALF[dt] + 2.0 ** -14 + (2.0 ** -25 * max(lk) if dt == F16 else 0.0)).all()


@pytest.mark.parametrize("kv,group,dt", [(2, 7, F16), (4, 16, BF16), (1, 1, BF16)])
def test_a_prompt_alone_and_in_batches(kv, group, dt):
    """Each sequence by itself, in batches of all kinds and in either order: how its work is cut, and so its last bits, may differ."""
    lq, lk = [300, 1, 77, 0, 1200, 16], [300, 2500, 900, 40, 1200, 3]
    q, k, v = (normal(91 + i, n, h, 128, dt=dt) for i, (n, h) in enumerate(((sum(lq), kv * group), (sum(lk), kv), (sum(lk), kv))))
    qs, ks, vs = q.split(lq), k.split(lk), v.split(lk)
    want = [paged.prompt(a.double(), b.double(), c.double(), [a.shape[0]], [b.shape[0]], SCALE) if a.shape[0] else None
            for a, b, c in zip(qs, ks, vs)]
    for batch in ([0], [1], [2], [4], [5], [0, 5], [5, 0, 2], [3, 0, 2, 5], [1, 4], list(range(6)), list(range(5, -1, -1)), [0, 2] * 40):
        m, n = [lq[s] for s in batch], [lk[s] for s in batch]
        out, lse, ws = _prompt(torch.cat([qs[s] for s in batch]), torch.cat([ks[s] for s in batch]), torch.cat([vs[s] for s in batch]), m, n)
        assert qsa.read_flags(ws) == 0
        for s, o, e in zip(batch, out.split(m), lse.split(m)):
            if lq[s]:
                check_attention(o, e, want[s], dt)


# ------------------------------------------------------------------ trees

def _tree_inputs(seed, n_tokens, nodes, kv, group, dt, spare=3):
    total = sum(nodes)
    q, k, v = normal(seed, total, kv * group, 128, dt=dt), normal(seed + 1, total, kv, 128, dt=dt), \
        normal(seed + 2, total, kv, 128, dt=dt, mean=0.25)
    pages = sum((n + 63) // 64 for n in n_tokens) + spare
    kc, vc = random_pool(seed + 3, kv, pages, dt)
    width = max((n + 63) // 64 for n in n_tokens) + 2
    return q, k, v, random_parents(seed, nodes), kc, vc, random_table(seed, n_tokens, pages, width)


def _tree(q, k, v, parents, nodes, kc, vc, table, n_tokens, out_dt=None, max_nodes=None, lse=True, scale=None):
    out = torch.full(q.shape, float("nan"), dtype=out_dt or q.dtype, device="cuda")
    ls = torch.full(q.shape[:2], float("nan"), device="cuda") if lse else None
    ws = qsa.alloc_attention_workspace(q.shape[0], q.shape[1], k.shape[1])
    qsa.tree_attention(q, k, v, i32(parents), i32(cu(nodes)), max_nodes or max(nodes), kc, vc, i32(table), i32(n_tokens), out, ls,
                       ws=ws, scale=scale)
    return out, ls, ws


def _want_tree(q, k, v, parents, nodes, kc, vc, table, n_tokens, scale=SCALE):
    return paged.tree(q.double(), k.double(), v.double(), parents, nodes, kc.double(), vc.double(), table, n_tokens, scale)


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("kv,group", [(4, 16), (2, 7), (1, 1), (2, 8)])
@pytest.mark.parametrize("n_tokens,nodes", [([0], [1]), ([1], [1]), ([63, 64, 65], [3, 1, 2]), ([500], [64]), ([0, 130, 1000], [5, 17, 33]),
                                            ([128], [16]), ([2000, 7], [1, 1])])
def test_tree_matches_the_definition(n_tokens, nodes, kv, group, dt):
    x = _tree_inputs(7, n_tokens, nodes, kv, group, dt)
    q, k, v, parents, kc, vc, table = x
    out, lse, ws = _tree(q, k, v, parents, nodes, kc, vc, table, n_tokens)
    check_attention(out, lse, _want_tree(q, k, v, parents, nodes, kc, vc, table, n_tokens), dt)
    assert qsa.read_flags(ws) == 0


@pytest.mark.parametrize("n_tokens,nodes,kv,group,dt", [
    ([9000], [1], 4, 16, BF16), ([12_345, 3, 700], [9, 64, 30], 2, 16, F16), ([100 * i for i in range(50)], [1 + i % 8 for i in range(50)], 2, 8, BF16),
    ([5000, 5000], [64, 64], 1, 16, BF16), ([3001], [61], 1, 13, F16)])
def test_tree_longer_and_ragged(n_tokens, nodes, kv, group, dt):
    q, k, v, parents, kc, vc, table = _tree_inputs(17, n_tokens, nodes, kv, group, dt)
    out, lse, ws = _tree(q, k, v, parents, nodes, kc, vc, table, n_tokens)
    check_attention(out, lse, _want_tree(q, k, v, parents, nodes, kc, vc, table, n_tokens), dt)
    assert qsa.read_flags(ws) == 0


def test_tree_empty_trees_fp32_output_and_a_loose_bound():
    n_tokens, nodes = [100, 50, 0, 300], [0, 4, 0, 2]
    q, k, v, parents, kc, vc, table = _tree_inputs(23, n_tokens, nodes, 2, 4, F16)
    out, lse, ws = _tree(q, k, v, parents, nodes, kc, vc, table, n_tokens, out_dt=torch.float32, max_nodes=64, scale=0.2)
    check_attention(out, lse, _want_tree(q, k, v, parents, nodes, kc, vc, table, n_tokens, 0.2), F16)
    out, lse, ws = _tree(q, k, v, parents, nodes, kc, vc, table, n_tokens, lse=False)
    check_attention(out, None, _want_tree(q, k, v, parents, nodes, kc, vc, table, n_tokens), F16)


@pytest.mark.parametrize("group", [1, 16])
def test_tree_unseen_rows_do_not_touch_it(group):
    """Page places behind the tokens, pages of others, and nodes that are no ancestors hold NaN or infinities."""
    n_tokens, nodes, kv = [100, 250], [6, 5], 2
    q, k, v, _, kc, vc, table = _tree_inputs(29, n_tokens, nodes, kv, group, BF16)
    parents = [-1, 0, 0, 1, 1, 2, -1, 0, 1, 2, 3]
    good, lse, _ = _tree(q, k, v, parents, nodes, kc, vc, table, n_tokens)
    for bad in (float("nan"), float("inf")):
        kc2, vc2 = torch.full_like(kc, bad), torch.full_like(vc, bad)
        for s, n in enumerate(n_tokens):
            for t in range(n):
                p = table[s][t // 64]
                kc2[:, 64 * p + t % 64], vc2[:, p, :, t % 64] = kc[:, 64 * p + t % 64], vc[:, p, :, t % 64]
        out, ls, ws = _tree(q, k, v, parents, nodes, kc2, vc2, table, n_tokens)
        assert torch.equal(out, good) and torch.equal(ls, lse) and qsa.read_flags(ws) == 0
        v2, k2 = v.clone(), k.clone()
        v2[2, :, 9] = bad          # node 2: its child 5 sees it, the others do not
        k2[4] = bad                # node 4: nobody but itself
        out, ls, _ = _tree(q, k2, v2, parents, nodes, kc, vc, table, n_tokens)
        for i in (0, 1, 3, 6, 7, 8, 9, 10):
            assert torch.equal(out[i], good[i]) and torch.equal(ls[i], lse[i])
        for i in (2, 5):
            assert not torch.isfinite(out[i, :, 9]).any()
            keep = [d for d in range(128) if d != 9]
            assert torch.equal(out[i][:, keep], good[i][:, keep])
        if math.isnan(bad):
            assert torch.isnan(out[4]).all()


def test_tree_bad_pages_parents_and_lengths_are_flagged():
    n_tokens, nodes, kv, group = [200, 300], [4, 3], 2, 4
    q, k, v, parents, kc, vc, table = _tree_inputs(31, n_tokens, nodes, kv, group, BF16)
    for bad in (-1, len(vc[0]), 2 ** 31 - 1, -2 ** 31):
        t2 = [list(r) for r in table]
        t2[0][1] = bad
        out, lse, ws = _tree(q, k, v, parents, nodes, kc, vc, t2, n_tokens)
        check_attention(out, lse, _want_tree(q, k, v, parents, nodes, kc, vc, t2, n_tokens), BF16)
        assert qsa.read_flags(ws) == qsa.FLAG_BAD_ID
    p2 = list(parents)
    p2[2], p2[5] = 2, 64
    out, lse, ws = _tree(q, k, v, p2, nodes, kc, vc, table, n_tokens)
    check_attention(out, lse, _want_tree(q, k, v, p2, nodes, kc, vc, table, n_tokens), BF16)
    assert qsa.read_flags(ws) == qsa.FLAG_BAD_ID
    good, _, _ = _tree(q, k, v, parents, nodes, kc, vc, table, n_tokens)
    out, lse, ws = _tree(q, k, v, parents, nodes, kc, vc, table, n_tokens, max_nodes=3)
    assert torch.equal(out[:3], good[:3]) and torch.isnan(out[3]).all() and torch.equal(out[4:], good[4:])
    assert qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED
    wide = 64 * len(table[0])
    out, lse, ws = _tree(q, k, v, parents, nodes, kc, vc, table, [-5, wide + 1])   # as 0 and the row's width
    assert qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED | qsa.FLAG_BAD_ID
    check_attention(out, lse, _want_tree(q, k, v, parents, nodes, kc, vc, table, [0, wide]), BF16)


@pytest.mark.parametrize("kv,group,dt", [(2, 7, F16), (8, 8, BF16)])
def test_a_tree_alone_and_in_batches(kv, group, dt):
    n_tokens, nodes = [900, 0, 64, 5000, 333], [3, 9, 1, 20, 64]
    q, k, v, parents, kc, vc, table = _tree_inputs(97, n_tokens, nodes, kv, group, dt)
    at = cu(nodes)
    want = _want_tree(q, k, v, parents, nodes, kc, vc, table, n_tokens)
    for batch in ([0], [1], [2], [3], [4], [0, 1], [3, 2, 0], list(range(5)), list(range(4, -1, -1))):
        rows = [i for s in batch for i in range(at[s], at[s + 1])]
        m = [nodes[s] for s in batch]
        out, lse, ws = _tree(q[rows], k[rows], v[rows], [parents[i] for i in rows], m, kc, vc, [table[s] for s in batch],
                             [n_tokens[s] for s in batch])
        check_attention(out, lse, [x[rows] for x in want], dt)
        assert qsa.read_flags(ws) == 0


def test_tree_of_one_node_is_the_last_row_of_a_prompt():
    """A decode step over pages against prompt attention with all the keys in rows."""
    n = 777
    q, k, v, parents, kc, vc, table = _tree_inputs(37, [n], [1], 2, 8, BF16)
    out, lse, _ = _tree(q, k, v, parents, [1], kc, vc, table, [n])
    pk, pv, _ = paged.paged_rows(kc, vc, table[0], n)
    out2, lse2, _ = _prompt(q, torch.cat((pk, k)), torch.cat((pv, v)), [1], [n + 1])
    want = _want_tree(q, k, v, parents, [1], kc, vc, table, [n])
    check_attention(out, lse, want, BF16)
    check_attention(out2, lse2, want, BF16)


def test_captured_calls_follow_their_inputs():
    """Captured once, replayed on new lengths, tables and values; on a stream of its own."""
    n_tokens, nodes, kv, group = [300, 90], [4, 3], 2, 8
    q, k, v, parents, kc, vc, table = _tree_inputs(41, n_tokens, nodes, kv, group, BF16)
    ws = qsa.alloc_attention_workspace(7, kv * group, kv)
    d = dict(parents=i32(parents), cu_nodes=i32(cu(nodes)), table=i32(table), n_tokens=i32(n_tokens))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    pout, plse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    cq, ck = i32([0, 4, 7]), i32([0, 4, 7])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        def step():
            qsa.tree_attention(q, k, v, d["parents"], d["cu_nodes"], 64, kc, vc, d["table"], d["n_tokens"], out, lse, ws=ws)
            qsa.prompt_attention(q, k, v, cq, ck, pout, plse, ws=ws)
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        for turn in range(3):
            nt, nn = ([300, 90], [64 + turn, 1])[turn % 2], ([4, 3], [2, 5])[turn % 2]
            par = random_parents(turn, nn)
            q.copy_(normal(50 + turn, *q.shape, dt=BF16))
            d["n_tokens"].copy_(i32(nt)), d["cu_nodes"].copy_(i32(cu(nn))), d["parents"].copy_(i32(par))
            ck.copy_(i32(cu(nn))), cq.copy_(i32(cu(nn)))
            g.replay()
            side.synchronize()
            check_attention(out, lse, _want_tree(q, k, v, par, nn, kc, vc, table, nt), BF16)
            check_attention(pout, plse, paged.prompt(q.double(), k.double(), v.double(), nn, nn, SCALE), BF16)
    assert qsa.read_flags(ws, stream=side) == 0


# ------------------------------------------------------------------ how the work is shared out

MANY = [(7 * i) % 41 for i in range(300)]            # with some of no queries
# (queries, keys, KV heads, group): runs in equal pieces; dealt out, by sequences in a warp and by more; cut at equal distances,
# by one long sequence and by more sequences than are counted
SHARED_OUT = [([40], [5000], 2, 16), ([300] * 20, [300 + 9 * i for i in range(20)], 4, 16),
              ([1 + i % 60 for i in range(200)], [70 + i for i in range(200)], 4, 8), ([4000, 30], [4000, 5000], 1, 16),
              (MANY, [m + 3 * (i % 30) for i, m in enumerate(MANY)], 2, 3),
              ([256], [8000], 4, 16), ([70, 250], [9000, 8200], 4, 15),
              ([0] * 299 + [1], [0] * 299 + [2000], 1, 16), ([0] * 270 + [5] + [0] * 20 + [40], [7] * 270 + [9000] + [0] * 20 + [1100], 2, 4)]


@pytest.mark.parametrize("lq,lk,kv,group", SHARED_OUT)
def test_prompt_however_its_runs_are_shared_out(lq, lk, kv, group):
    _check_prompt(lq, lk, kv, group, BF16, seed=5)


TREES = [([3000, 10, 500], [40, 64, 3], 1, 16), ([300 + 20 * i for i in range(20)], [1 + 3 * i for i in range(20)], 4, 16),
         ([10 * i for i in range(60)], [1 + i % 33 for i in range(60)], 2, 16), ([9000] + [100] * 40, [50] * 41, 2, 13),
         ([5 * i for i in range(300)], [(5 * i) % 9 for i in range(300)], 1, 8), ([2 * i for i in range(300)], [1] * 300, 2, 16),
         ([0] * 299 + [1500], [0] * 299 + [1], 1, 16), ([0] * 260 + [3000, 0, 500], [0] * 260 + [60, 0, 9], 2, 5)]


@pytest.mark.parametrize("n_tokens,nodes,kv,group", TREES)
def test_tree_however_its_runs_are_shared_out(n_tokens, nodes, kv, group):
    q, k, v, parents, kc, vc, table = _tree_inputs(61, n_tokens, nodes, kv, group, BF16)
    out, lse, ws = _tree(q, k, v, parents, nodes, kc, vc, table, n_tokens)
    check_attention(out, lse, _want_tree(q, k, v, parents, nodes, kc, vc, table, n_tokens), BF16)
    assert qsa.read_flags(ws) == 0


def test_one_workspace_serves_calls_of_every_kind():
    """Prompts and trees of all kinds in turn, twice: each leaves the workspace as the next one needs it."""
    ws = qsa.alloc_attention_workspace(6100, 64, 4)
    calls = []
    for i, (lq, lk, kv, group) in enumerate(SHARED_OUT):
        q, k, v = normal(i, sum(lq), kv * group, 128, dt=BF16), *(normal(9 + i, sum(lk), kv, 128, dt=BF16) for _ in "kv")
        calls.append((lambda out, ls, w, a=(q, k, v, i32(cu(lq)), i32(cu(lk))): qsa.prompt_attention(*a, out, ls, ws=w), q, kv))
        if i < len(TREES):
            n_tokens, nodes, kv, group = TREES[i]
            q, k, v, parents, kc, vc, table = _tree_inputs(71 + i, n_tokens, nodes, kv, group, BF16)
            a = (q, k, v, i32(parents), i32(cu(nodes)), max(nodes), kc, vc, i32(table), i32(n_tokens))
            calls.append((lambda out, ls, w, a=a: qsa.tree_attention(*a, out, ls, ws=w), q, kv))
    first = []
    for call, q, kv in calls:
        out, ls = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        call(out, ls, qsa.alloc_attention_workspace(q.shape[0], q.shape[1], kv))
        first.append((out, ls))
    for _ in range(2):
        for (call, q, _), (want, lse) in zip(calls, first):
            out, ls = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device="cuda")
            call(out, ls, ws)
            assert torch.equal(out, want) and torch.equal(ls, lse)
    assert qsa.read_flags(ws) == 0


def test_two_streams_with_a_workspace_each():
    lens, kv, group = [700, 40, 900], 2, 16
    q, k, v = (normal(i, sum(lens), h, 128, dt=BF16) for i, h in ((1, kv * group), (2, kv), (3, kv)))
    want, lse, _ = _prompt(q, k, v, lens, lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [qsa.alloc_attention_workspace(sum(lens), kv * group, kv) for _ in streams]
    outs = [[torch.full_like(q, float("nan")) for _ in range(4)] for _ in streams]
    c = i32(cu(lens))
    torch.cuda.synchronize()
    for i in range(4):
        for st, ws, out in zip(streams, spaces, outs):
            qsa.prompt_attention(q, k, v, c, c, out[i], ws=ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for out in outs for x in out)


def test_a_captured_prompt_follows_its_lengths_from_kind_to_kind():
    total, keys, kv, group = 2600, 5200, 1, 16
    q, k, v = normal(1, total, kv * group, 128, dt=BF16), *(normal(2 + i, keys, kv, 128, dt=BF16) for i in range(2))
    cq, ck = i32([0] * 21), i32([0] * 21)
    ws = qsa.alloc_attention_workspace(total, kv * group, kv)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    qsa.prompt_attention(q, k, v, cq, ck, out, lse, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qsa.prompt_attention(q, k, v, cq, ck, out, lse, ws=ws)
    for lq, lk in (([50], [5000]), ([130] * 20, [260] * 20), ([2600], [5200]), ([0, 0, 7], [0, 3, 2000]), ([130] * 20, [130] * 20)):
        cq.copy_(i32(cu(lq + [0] * (20 - len(lq))))), ck.copy_(i32(cu(lk + [0] * (20 - len(lk)))))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        n, m = sum(lq), sum(lk)
        check_attention(out[:n], lse[:n], paged.prompt(q[:n].double(), k[:m].double(), v[:m].double(), lq, lk, SCALE), BF16)
        assert torch.isnan(out[n:]).all()
    assert qsa.read_flags(ws) == 0


@pytest.mark.parametrize("group,long", [(16, 5000), (3, 700), (16, 300)])
def test_a_large_tree_is_not_touched_by_what_it_does_not_see(group, long):
    """Two streams of rows, several tiles of them, a run in pieces: NaN behind the tokens and in nodes that are no ancestors."""
    n_tokens, nodes, kv = [long, 77], [60, 44], 2
    q, k, v, _, kc, vc, table = _tree_inputs(83, n_tokens, nodes, kv, group, BF16)
    parents = [i - 2 if i >= 2 else -1 for m in nodes for i in range(m)]     # two paths: the even nodes and the odd ones
    good, lse, _ = _tree(q, k, v, parents, nodes, kc, vc, table, n_tokens)
    kc2, vc2 = torch.full_like(kc, float("nan")), torch.full_like(vc, float("nan"))
    for s, n in enumerate(n_tokens):
        for j in range((n + 63) // 64):
            p, m = table[s][j], min(64, n - 64 * j)
            kc2[:, 64 * p:64 * p + m], vc2[:, p, :, :m] = kc[:, 64 * p:64 * p + m], vc[:, p, :, :m]
    for first in (0, 60):
        k2, v2 = k.clone(), v.clone()
        v2[first + 31] = float("inf")
        k2[first + 33] = float("nan")
        out, ls, ws = _tree(q, k2, v2, parents, nodes, kc2, vc2, table, n_tokens)
        touched = torch.zeros(104, dtype=torch.bool)
        touched[first + 31:first + nodes[first > 0]:2] = True
        assert torch.equal(out[~touched], good[~touched]) and torch.equal(ls[~touched], lse[~touched])
        assert not torch.isfinite(out[touched]).any() and torch.isnan(ls[first + 33]).all()
        assert qsa.read_flags(ws) == 0


def test_a_chunk_cut_in_pieces_is_not_touched_by_what_it_does_not_see():
    """A run's last, masked step need not be the last one that its CTA works on."""
    lq, lk, kv, group = 256, 8000, 4, 16
    q, k, v = normal(1, lq, kv * group, 128, dt=BF16), normal(2, lk, kv, 128, dt=BF16), normal(3, lk, kv, 128, dt=BF16)
    good, lse, _ = _prompt(q, k, v, [lq], [lk])
    for row in (1, 100, 255):                    # of the last 256 keys, seen from this query on
        for bad in (float("nan"), -float("inf")):
            k2, v2 = k.clone(), v.clone()
            k2[lk - lq + row + 1:] = bad
            v2[lk - lq + row, 1] = bad
            out, ls, ws = _prompt(q, k2, v2, [lq], [lk])
            assert torch.equal(out[:row], good[:row]) and torch.equal(ls[:row], lse[:row])
            other = [h for h in range(kv * group) if h // group != 1]
            assert torch.equal(out[row][other], good[row][other]) and torch.equal(ls[row], lse[row])
            assert not torch.isfinite(out[row, group:2 * group]).any()
            assert qsa.read_flags(ws) == 0
