"""Eviction on the GPU against the oracle: block weights added up, the plan, the moved records, and
the whole loop of a decode with eviction."""
import numpy as np
import pytest

from oracle import qcache as oq

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_kv_gb300 import qsa  # noqa: E402

from .qcache_cases import DT, check_attention, random_cache, random_ids, to16  # noqa: E402


def _ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# ------------------------------------------------------------------ weights

@pytest.mark.parametrize("nq,kv,k,n", [(1, 1, 1, 1), (3, 4, 32, 4032), (256, 4, 32, 8125), (7, 2, 64, 100), (1000, 8, 5, 513),
                                       (2, 1, 9, 100_000), (1024, 8, 64, 16_384), (5, 3, 17, 511)])
@pytest.mark.parametrize("prev", [False, True])
def test_weights_add_matches_the_oracle(nq, kv, k, n, prev):
    """Each weight is held to 2^-37, the sum and the decay in 64 bits, the result rounded once."""
    rng = np.random.default_rng(nq + k)
    w = (rng.random((nq, kv, k)) ** 4 * 16).astype(np.float32)
    w[rng.random(w.shape) < 0.1] = 0
    ids = rng.integers(0, n, size=(nq, k)).astype(np.int32)          # repeats within and across queries
    ids[rng.random(ids.shape) < 0.2] = -1
    p = (rng.random(n) * 50).astype(np.float32)
    decay = 0.9375
    ws = _ws()
    acc = torch.full((n,), float("nan"), device="cuda")
    qsa.block_weights_add(_cuda(w), _cuda(ids), acc, prev=_cuda(p) if prev else None, decay=decay, ws=ws)
    want = oq.weights_add(w, ids, decay, p if prev else None, n)
    bound = nq * kv * k * 2.0 ** -37 / max(1, n) * 64 + 2.0 ** -24 * np.abs(want) + 1e-9
    assert (np.abs(acc.cpu().double().numpy() - want) <= bound).all()
    assert qsa.read_flags(ws) == 0
    again = torch.empty_like(acc)
    qsa.block_weights_add(_cuda(w), _cuda(ids), again, prev=_cuda(p) if prev else None, decay=decay)
    assert torch.equal(acc, again)
    order = rng.permutation(nq)                                       # the order of the queries changes nothing
    qsa.block_weights_add(_cuda(w[order]), _cuda(ids[order]), again, prev=_cuda(p) if prev else None, decay=decay)
    assert torch.equal(acc, again)


def test_weights_add_in_place_and_bad_values():
    n = 700
    w = torch.ones(2, 1, 4, device="cuda")
    ids = torch.tensor([[0, 5, 699, -1], [5, 5, 0, 3]], dtype=torch.int32, device="cuda")
    acc = torch.full((n,), 2.0, device="cuda")
    ws = _ws()
    qsa.block_weights_add(w, ids, acc, prev=acc, decay=0.5, ws=ws)
    want = np.ones(n)
    want[[0, 5, 699, 3]] += [2, 3, 1, 1]
    np.testing.assert_array_equal(acc.cpu().numpy(), want)
    assert qsa.read_flags(ws) == 0
    w = torch.tensor([[[float("nan"), float("inf"), -1.0, 33.0]]], device="cuda")
    qsa.block_weights_add(w, torch.tensor([[1, 2, 3, 4]], dtype=torch.int32, device="cuda"), acc, ws=ws)
    assert acc[:6].tolist() == [0.0, 0.0, 32.0, 0.0, 32.0, 0.0]
    assert qsa.read_flags(ws) == qsa.FLAG_BAD_WEIGHT
    ids = torch.tensor([[700, -2, 1, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    qsa.block_weights_add(torch.ones(1, 1, 4, device="cuda"), ids, acc, ws=ws)
    assert acc.sum().item() == 1.0 and acc[1].item() == 1.0
    assert qsa.read_flags(ws) == qsa.FLAG_BAD_ID


def test_weights_add_largest_sum():
    """2^22 weights of 32 on one block: the integer sum stays in 64 bits."""
    w = torch.full((1 << 13, 8, 64), 32.0, device="cuda")
    ids = torch.full((1 << 13, 64), 1, dtype=torch.int32, device="cuda")
    acc = torch.empty(3, device="cuda")
    qsa.block_weights_add(w, ids, acc)
    assert acc.tolist() == [0.0, 2.0 ** 27, 0.0]


# ------------------------------------------------------------------ plan

@pytest.mark.parametrize("n,keep,first,last", [(1, 1, 0, 1), (64, 16, 1, 1), (257, 128, 1, 8), (1024, 1023, 0, 1),
                                               (1025, 5, 4, 1), (8125, 4096, 4, 64), (8192, 1, 0, 1), (40_000, 20_001, 10, 300),
                                               (300, 300, 5, 7), (5000, 4999, 2500, 2499),
                                               (2048, 777, 2, 3), (2049, 2000, 2, 3), (4096, 4000, 1, 1), (4097, 17, 4, 4),
                                               (8193, 8000, 1, 1), (16_384, 9_999, 3, 50), (16_385, 100, 0, 1)])
@pytest.mark.parametrize("kind", ["random", "levels", "equal", "special"])
def test_plan_matches_the_oracle(n, keep, first, last, kind):
    rng = np.random.default_rng(n + keep)
    w = (rng.random(n) ** 6 * 100).astype(np.float32)
    if kind == "levels":
        w = np.floor(w / 10).astype(np.float32) * np.where(rng.random(n) < 0.5, -1, 1).astype(np.float32)   # -0 among them
    elif kind == "equal":
        w[:] = 3
    elif kind == "special":
        w[rng.random(n) < 0.1] = np.nan
        w[rng.random(n) < 0.05] = np.inf
        w[rng.random(n) < 0.05] = -np.inf
        w[rng.random(n) < 0.3] = 0
        w[rng.random(n) < 0.1] = 1e-42                               # subnormal
    for tokens in (64 * n, 64 * n - 63, max(1, 64 * (n // 2) + 5), 1, 0):
        out = torch.full((1, keep), -7, dtype=torch.int32, device="cuda")
        new = torch.full((1,), -7, dtype=torch.int32, device="cuda")
        ws = _ws()
        qsa.evict_plan(_cuda(w[None]), torch.tensor([tokens], dtype=torch.int32, device="cuda"), out, new, first, last, ws=ws)
        kept, left = oq.evict_plan(w, tokens, keep, first, last)
        np.testing.assert_array_equal(out.cpu().numpy()[0], kept)
        assert new.item() == left and qsa.read_flags(ws) == 0


def test_plan_of_many_rows_with_a_stride_and_clamps():
    rng = np.random.default_rng(1)
    rows, n, keep = 70, 500, 200
    w = rng.random((rows, 640)).astype(np.float32)
    nt = rng.integers(0, 64 * n + 1, size=rows).astype(np.int32)
    out = torch.empty(rows, keep, dtype=torch.int32, device="cuda")
    new = torch.empty(rows, dtype=torch.int32, device="cuda")
    ws = _ws()
    d = _cuda(w)[:, :n]
    qsa.evict_plan(d, _cuda(nt), out, new, 3, 10, ws=ws)
    assert qsa.read_flags(ws) == 0
    for r in range(rows):
        kept, left = oq.evict_plan(w[r, :n], int(nt[r]), keep, 3, 10)
        np.testing.assert_array_equal(out[r].cpu().numpy(), kept)
        assert new[r].item() == left
    nt[3], nt[5] = -1, 64 * n + 1
    qsa.evict_plan(d, _cuda(nt), out, new, 3, 10, ws=ws)
    assert qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED
    assert (out[3] == -1).all() and new[3].item() == 0
    kept, left = oq.evict_plan(w[5, :n], 64 * n, keep, 3, 10)
    np.testing.assert_array_equal(out[5].cpu().numpy(), kept)
    assert new[5].item() == left


def test_plan_of_a_very_long_row():
    n, keep = 3_000_000, 1_234_567
    w = torch.rand(1, n, device="cuda").pow_(3)
    w[0, ::3] = 0.25                                                  # a million ties
    out = torch.empty(1, keep, dtype=torch.int32, device="cuda")
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    qsa.evict_plan(w, torch.tensor([64 * n - 9], dtype=torch.int32, device="cuda"), out, new, 100, 1000)
    key = w[0].clone()
    key[:100] = key[n - 1000:] = float("inf")
    want = key.sort(descending=True, stable=True).indices[:keep].sort().values
    assert torch.equal(out[0].long(), want) and new.item() == 64 * keep - 9


# ------------------------------------------------------------------ move

def test_gather_moves_records_of_every_size():
    rng = np.random.default_rng(2)
    blocks, slots, n = 50, 30, 21
    keep = np.full(n, -1, dtype=np.int32)
    keep[:19] = np.sort(rng.permutation(blocks)[:19])
    keep[7] = -1
    shapes = [((3, blocks, oq.REC), torch.uint8), ((blocks, 128), torch.bfloat16), ((blocks,), torch.float32),
              ((2, blocks, 64 * 128), torch.float16), ((2, blocks, 128, 64), torch.bfloat16), ((blocks, 3), torch.float32),
              ((5, blocks, 4), torch.uint8), ((blocks, 128), torch.float32)]
    pairs, want = [], []
    for i, (shape, dt) in enumerate(shapes):
        src = torch.randint(0, 255, shape + (torch.empty(0, dtype=dt).element_size(),), dtype=torch.uint8, device="cuda")
        src = src.flatten(-2).view(dt).view(shape)
        at = 1 if len(shape) >= 3 else 0
        dst = torch.randint(0, 255, shape[:at] + (slots,) + shape[at + 1:], device="cuda").to(dt)
        ref = dst.clone()
        for j, b in enumerate(keep):
            if b >= 0:
                ref.select(at, j).copy_(src.select(at, int(b)))
        pairs.append((src, dst))
        want.append(ref)
    ws = _ws()
    qsa.gather_blocks(pairs, _cuda(keep), ws=ws)
    for (_, dst), ref in zip(pairs, want):
        assert torch.equal(dst.reshape(-1).view(torch.uint8), ref.reshape(-1).view(torch.uint8))
    assert qsa.read_flags(ws) == 0
    keep[3], keep[4] = blocks, -5
    qsa.gather_blocks(pairs, _cuda(keep), ws=ws)
    for (_, dst), ref in zip(pairs, want):
        assert torch.equal(dst.reshape(-1).view(torch.uint8), ref.reshape(-1).view(torch.uint8))   # bad ids: left as they were
    assert qsa.read_flags(ws) == qsa.FLAG_BAD_ID


def test_gather_of_unaligned_arrays():
    """Bases at 4 bytes past a 16-byte boundary, records of 16 and of 20 bytes."""
    x = torch.randint(0, 255, (4 + 16 * 40,), dtype=torch.uint8, device="cuda")
    y = torch.zeros(4 + 16 * 40, dtype=torch.uint8, device="cuda")
    z = torch.randint(0, 1 << 30, (33, 5), dtype=torch.int32, device="cuda")
    zd = torch.zeros(12, 5, dtype=torch.int32, device="cuda")
    keep = torch.arange(0, 24, 2, dtype=torch.int32, device="cuda")
    qsa.gather_blocks([(x[4:].view(40, 16), y[4:].view(40, 16)), (z, zd)], keep)
    assert torch.equal(y[4:].view(40, 16)[:12], x[4:].view(40, 16)[:24:2]) and not y[4:].view(40, 16)[12:].any()
    assert torch.equal(zd, z[:24:2])


def test_gather_past_four_gigabytes():
    src = torch.zeros(1, 500_000, oq.REC, dtype=torch.uint8, device="cuda")
    ids = [3, 250_001, 494_000, 499_999]
    for i, b in enumerate(ids):
        src[0, b] = i + 1
    dst = torch.zeros(1, 500_000, oq.REC, dtype=torch.uint8, device="cuda")
    keep = torch.full((500_000,), -1, dtype=torch.int32, device="cuda")
    at = [0, 100, 494_500, 499_998]
    keep[at] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    qsa.gather_blocks([(src, dst)], keep)
    for i, b in enumerate(at):
        assert (dst[0, b] == i + 1).all()
        dst[0, b] = 0
    assert not dst.any()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt", [oq.BF16, oq.F16])
def test_select_attend_accumulate_and_evict_together(fmt):
    """A prompt written to a 4-bit cache; decode steps that append, select, attend and accumulate;
    the cache evicted to half its blocks with its indexer keys; and attention over what is left:
    everything against the oracle on the same bytes."""
    rng = np.random.default_rng(3)
    kv, group, blocks, k, tokens = 2, 16, 40, 8, 33 * 64 + 17
    heads = kv * group
    cache = qsa.alloc_qcache(kv, 64 * blocks)
    kr, _ = to16(rng.normal(size=(tokens, kv, 128)), fmt)
    vr, _ = to16(rng.normal(size=(tokens, kv, 128)), fmt)
    qsa.qcache_append(kr, vr, cache, 0)
    kblk = torch.randn(blocks, 128, device="cuda").bfloat16()
    acc = torch.zeros(blocks, device="cuda")
    n = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    ws, sel = _ws(), qsa.alloc_workspace(1, blocks, k)
    want_acc = np.zeros(blocks)
    scale = float(np.float32(128 ** -0.5))
    for step in range(4):
        kr, _ = to16(rng.normal(size=(1, kv, 128)), fmt)
        vr, _ = to16(rng.normal(size=(1, kv, 128)), fmt)
        qsa.qcache_append(kr, vr, cache, n, ws=ws)
        n += 1
        nb = (n + 63) // 64
        iq, iw = torch.randn(1, 16, 128, device="cuda").bfloat16(), torch.rand(1, 16, device="cuda")
        ids = torch.empty(1, k, dtype=torch.int32, device="cuda")
        qsa.select(iq, iw, kblk, nb, k, ids, sel, scores=torch.empty(1, blocks, device="cuda"))
        q, qd = to16(rng.normal(size=(1, heads, 128)) * 2, fmt)
        out, lse = torch.empty_like(q), torch.empty(1, heads, device="cuda")
        w = torch.empty(1, kv, k, device="cuda")
        qsa.select_attention_qcache(q, cache, ids, n, out, lse, w, ws=ws)
        qsa.block_weights_add(w, ids, acc, prev=acc, decay=0.75, ws=ws)
        host, hid = cache.cpu().numpy(), ids.cpu().numpy()
        want = oq.attention(qd, host, hid, n.cpu().numpy(), scale, fmt)
        check_attention([t.double().cpu().numpy() for t in (out, lse, w)], want, fmt)
        want_acc = oq.weights_add(want[2], hid, 0.75, want_acc, blocks)
        np.testing.assert_allclose(acc.cpu().numpy(), want_acc, rtol=1e-3, atol=1e-6)
    n_keep = 20
    keep = torch.empty(1, n_keep, dtype=torch.int32, device="cuda")
    left = torch.empty(1, dtype=torch.int32, device="cuda")
    qsa.evict_plan(acc[None], n, keep, left, n_first=1, n_last=3, ws=ws)
    small = qsa.alloc_qcache(kv, 64 * 24)
    skblk, sacc = torch.zeros(24, 128, device="cuda").bfloat16(), torch.zeros(24, device="cuda")
    qsa.gather_blocks([(cache, small), (kblk, skblk), (acc, sacc)], keep[0], ws=ws)
    kept, tokens_left = oq.evict_plan(acc.cpu().numpy(), int(n.item()), n_keep, 1, 3)
    np.testing.assert_array_equal(keep.cpu().numpy()[0], kept)
    assert left.item() == tokens_left == n.item() - 64 * (34 - n_keep)
    assert torch.equal(small[:, :n_keep], cache[:, kept.tolist()]) and not small[:, n_keep:].any()
    assert torch.equal(skblk[:n_keep], kblk[kept.tolist()]) and torch.equal(sacc[:n_keep], acc[kept.tolist()])
    # the step goes on over the evicted cache: the same attention as over the kept blocks of the old one
    q, qd = to16(rng.normal(size=(1, heads, 128)), fmt)
    new_ids = torch.tensor([[0, 4, 11, 17, 18, 19, -1, -1]], dtype=torch.int32, device="cuda")
    old_ids = torch.where(new_ids >= 0, keep[0, new_ids.clamp(min=0).long()], -1).int()
    res = []
    for c, i, m in ((small, new_ids, left), (cache, old_ids, n)):
        o, w = torch.empty_like(q), torch.empty(1, kv, k, device="cuda")
        qsa.select_attention_qcache(q, c, i, m, o, None, w, ws=ws)
        res.append((o, w))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    check_attention([res[0][0].double().cpu().numpy(), None, None],
                    oq.attention(qd, small.cpu().numpy(), new_ids.cpu().numpy(), left.cpu().numpy(), scale, fmt), fmt)
    assert qsa.read_flags(ws) == 0


def test_captured_loop_with_eviction_shares_one_workspace():
    """Two captured graphs that use one workspace, replayed in turn, against eager calls."""
    fmt, kv, blocks, k, n_keep = oq.BF16, 2, 64, 16, 32
    cache = torch.from_numpy(random_cache(4, kv, blocks, fmt)).cuda()
    nt = torch.full((2,), 64 * blocks - 20, dtype=torch.int32, device="cuda")
    ws = _ws()
    steps = []
    for seed in (5, 6):
        q, _ = to16(np.random.default_rng(seed).normal(size=(2, 32, 128)), fmt)
        ids = _cuda(random_ids(seed, 2, k, np.full(2, 64 * blocks - 20)))
        steps.append(dict(q=q, ids=ids, out=torch.empty_like(q), w=torch.empty(2, kv, k, device="cuda"),
                          acc=torch.zeros(blocks, device="cuda"), keep=torch.empty(1, n_keep, dtype=torch.int32, device="cuda"),
                          left=torch.empty(1, dtype=torch.int32, device="cuda"), dst=qsa.alloc_qcache(kv, 64 * n_keep)))

    def call(s):
        qsa.select_attention_qcache(s["q"], cache, s["ids"], nt, s["out"], None, s["w"], ws=ws)
        qsa.block_weights_add(s["w"], s["ids"], s["acc"], prev=s["acc"], decay=0.5, ws=ws)
        qsa.evict_plan(s["acc"][None], nt[:1], s["keep"], s["left"], 1, 4, ws=ws)
        qsa.gather_blocks([(cache, s["dst"])], s["keep"][0], ws=ws)

    for s in steps:
        call(s)
    torch.cuda.synchronize()
    want = [{n: t.clone() for n, t in s.items()} for s in steps]
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(s)
        graphs.append(g)
    for _ in range(3):
        for s, g in zip(steps, graphs):
            for n in ("acc", "out", "w", "keep", "left", "dst"):
                s[n].zero_()
            g.replay()
    torch.cuda.synchronize()
    for s, x in zip(steps, want):
        for n in x:
            assert torch.equal(s[n], x[n]), n
    assert qsa.read_flags(ws) == 0


@pytest.mark.parametrize("n,keep", [(257, 128), (1024, 500), (2000, 1999), (4096, 100), (8125, 4096), (12_000, 5000), (17_000, 6000)])
def test_plan_updates_the_lengths_in_place(n, keep):
    """new_tokens is n_tokens, row after row, for every kernel of the plan: ids and lengths as out of place."""
    rng = np.random.default_rng(n)
    rows = 300
    w = torch.rand(rows, n, device="cuda")
    tokens = rng.integers(0, 64 * n + 1, size=rows).astype(np.int32)
    tokens[::3] = 64 * keep + rng.integers(-64, 129, size=len(tokens[::3]))   # just all of them kept, or just not
    tokens = np.minimum(tokens, 64 * n)
    nt = _cuda(tokens)
    keeps = [torch.empty(rows, keep, dtype=torch.int32, device="cuda") for _ in range(2)]
    left = torch.empty(rows, dtype=torch.int32, device="cuda")
    qsa.evict_plan(w, nt, keeps[0], left, 3, 10)
    for _ in range(5):
        there = nt.clone()
        keeps[1].fill_(-7)
        qsa.evict_plan(w, there, keeps[1], there, 3, 10)
        assert torch.equal(there, left) and torch.equal(keeps[0], keeps[1])
    for r in range(0, rows, 37):
        kept, want = oq.evict_plan(w[r].cpu().numpy(), int(tokens[r]), keep, 3, 10)
        np.testing.assert_array_equal(keeps[1][r].cpu().numpy(), kept)
        assert there[r].item() == want


@pytest.mark.parametrize("nq", [3, 100])
@pytest.mark.parametrize("decay", [0.98, 0.9, 1 / 3])
def test_weights_add_keeps_the_decay_in_64_bits(decay, nq):
    """A decay that fp32 does not hold: decay * prev + sum in 64 bits, rounded once (the weights are whole numbers, so
    their sum is exact, and numpy forms the same two roundings)."""
    rng = np.random.default_rng(int(decay * 100))
    n = 5000
    prev = (rng.random(n) * 50).astype(np.float32)
    ids = rng.integers(0, n, size=(nq, 16)).astype(np.int32)
    w = rng.integers(0, 17, size=(nq, 2, 16)).astype(np.float32)
    add = np.zeros(n)
    np.add.at(add, ids.reshape(-1), w.sum(1, dtype=np.float64).reshape(-1))
    acc = torch.empty(n, device="cuda")
    qsa.block_weights_add(_cuda(w), _cuda(ids), acc, prev=_cuda(prev), decay=decay)
    double = decay * prev.astype(np.float64) + add
    got = acc.cpu().numpy()
    # one rounding to fp32 of a double that is at most one step of 2^-53 off (a product and a sum, or both in one)
    assert (np.abs(got - double) <= np.abs(double) * (2.0 ** -24 + 2.0 ** -52)).all()
    assert (got == double.astype(np.float32)).mean() > 0.999


def test_captured_on_several_streams():
    """One captured graph that forks: the append on one stream, attention and weights on another behind it, the plan on
    a third, and the move behind all of them; replays give what eager calls give."""
    fmt, kv, blocks, k, n_keep = oq.BF16, 2, 40, 8, 16
    start = torch.from_numpy(random_cache(8, kv, blocks, fmt)).cuda()
    rng = np.random.default_rng(9)
    rows = [to16(rng.normal(size=(3, kv, 128)), fmt)[0] for _ in "kv"]
    q, _ = to16(rng.normal(size=(2, 32, 128)), fmt)
    ids = _cuda(random_ids(9, 2, k, np.full(2, 64 * blocks - 70)))
    src = torch.rand(blocks, device="cuda")

    def buffers():
        return dict(cache=start.clone(), n=torch.tensor([64 * blocks - 70] * 2, dtype=torch.int32, device="cuda"),
                    out=torch.zeros_like(q), w=torch.zeros(2, kv, k, device="cuda"), acc=torch.zeros(blocks, device="cuda"),
                    keep=torch.zeros(1, n_keep, dtype=torch.int32, device="cuda"), left=torch.zeros(1, dtype=torch.int32, device="cuda"),
                    dst=torch.zeros(kv, n_keep, oq.REC, dtype=torch.uint8, device="cuda"), low=torch.zeros(n_keep, device="cuda"))

    def step(b, side, third):
        main = torch.cuda.current_stream()
        qsa.qcache_append(*rows, b["cache"], b["n"][:1])
        b["n"] += 3
        side.wait_stream(main)
        third.wait_stream(main)
        with torch.cuda.stream(third):                     # the plan by weights at hand, beside the attention
            qsa.evict_plan(src[None], b["n"][:1], b["keep"], b["left"], 1, 2)
        with torch.cuda.stream(side):
            qsa.select_attention_qcache(q, b["cache"], ids, b["n"], b["out"], None, b["w"])
            qsa.block_weights_add(b["w"], ids, b["acc"], prev=b["acc"], decay=0.75)
        main.wait_stream(side)
        main.wait_stream(third)
        qsa.gather_blocks([(b["cache"], b["dst"]), (b["acc"], b["low"])], b["keep"][0])

    want, got = buffers(), buffers()
    s = torch.cuda.current_stream()
    for _ in range(3):
        step(want, s, s)
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(got, side, third)
    for name, x in buffers().items():
        got[name].copy_(x)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name
