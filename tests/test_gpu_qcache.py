"""The 4-bit KV cache on the GPU against the FP64 oracle: the writer byte for byte, the reader, and
selection attention over it, within bounds made of their roundings (tests/qcache_cases.py)."""
import numpy as np
import pytest

from oracle import qcache as oq

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_kv_gb300 import qsa  # noqa: E402

from .qcache_cases import DT, check_attention, random_cache, random_ids, to16  # noqa: E402

FMTS = [oq.BF16, oq.F16]


def _ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ writer and reader

def _rows(seed, n, kv):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(n, kv, 128))
    x[:, :, ::31] *= 6
    x += rng.normal(size=(n, kv, 1)) * 2
    return x


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,first,kv,blocks", [(1, 0, 1, 1), (1, 95, 3, 2), (63, 1, 2, 2), (64, 64, 1, 3), (65, 63, 2, 3),
                                               (200, 37, 4, 5), (5, 187, 2, 3), (384, 0, 1, 6)])
def test_append_writes_the_oracles_bytes(n, first, kv, blocks, fmt):
    """Over a cache of random bytes: the range's bytes are the oracle's, all others keep theirs."""
    k, kd = to16(_rows(10 * n + first, n, kv), fmt)
    v, vd = to16(_rows(10 * n + first + 1, n, kv), fmt)
    want = np.random.default_rng(n).integers(0, 256, size=(kv, blocks, oq.REC), dtype=np.uint8)
    cache = torch.from_numpy(want).cuda()
    ws = _ws()
    qsa.qcache_append(k, v, cache, first, ws=ws)
    oq.append(want, kd, vd, first, fmt)
    np.testing.assert_array_equal(cache.cpu().numpy(), want)
    assert qsa.read_flags(ws) == 0
    ko, vo = torch.full_like(k, 7), torch.full_like(v, 7)
    qsa.qcache_load(cache, ko, vo, first)
    rk, rv = oq.rows(want, first, n, fmt)
    for got, ref in ((ko, rk), (vo, rv)):   # fp64 to fp32 is exact here: 8 or 11 bits times 4, plus one 16-bit value
        assert torch.equal(got.cpu(), torch.from_numpy(ref).float().to(DT[fmt]))


@pytest.mark.parametrize("fmt", FMTS)
def test_append_special_rows(fmt):
    """Constant and zero rows, wide offsets, tiny ranges, exact ties, subnormal scales, the
    format's largest values, and rows with an infinity or a NaN."""
    rng = np.random.default_rng(5)
    big = 65504.0 if fmt == oq.F16 else 3.0e38
    rows = [np.zeros(128), np.full(128, -2.5), 1000 + rng.integers(0, 5, 128), rng.integers(0, 16, 128) + 0.0,
            rng.integers(0, 31, 128) / 2.0, rng.integers(0, 61, 128) / 4.0 - 8, rng.normal(size=128) * 1e-6,
            rng.normal(size=128) * 6e-8, rng.integers(0, 3, 128) * 6e-8, rng.uniform(-1, 1, 128) * big / 4,
            np.where(rng.random(128) < 0.5, big, 0.0), np.where(rng.random(128) < 0.5, -big, big),
            np.where(np.arange(128) == 9, np.inf, 1.0), np.where(np.arange(128) == 100, -np.inf, 1.0),
            np.where(np.arange(128) == 3, np.nan, rng.normal(size=128)), np.full(128, np.nan),
            np.where(np.arange(128) == 0, -7.0, 2.0 ** -11 * rng.integers(0, 9, 128)),
            np.where(np.arange(128) == 5, 30.0, rng.normal(size=128) * 2.0 ** -9)]
    with np.errstate(over="ignore", invalid="ignore"):
        k, kd = to16(np.stack(rows)[:, None], fmt)
    v, vd = k.flip(0), kd[::-1].copy()
    cache = torch.zeros(1, 1, oq.REC, dtype=torch.uint8, device="cuda")
    qsa.qcache_append(k, v, cache, 11)
    want = np.zeros((1, 1, oq.REC), dtype=np.uint8)
    oq.append(want, kd, vd, 11, fmt)
    np.testing.assert_array_equal(cache.cpu().numpy(), want)


def test_append_ties_and_near_ties_of_many_scales():
    """Rows of few-bit values: quotients on and beside the half-way points, for many scales."""
    rng = np.random.default_rng(6)
    n = 640
    x = rng.integers(-40, 41, size=(n, 1, 128)) * np.exp2(rng.integers(-6, 7, size=(n, 1, 1)).astype(float))
    x[::3] += np.exp2(rng.integers(-3, 9, size=(len(x[::3]), 1, 1)).astype(float))
    x[1::5, :, :8] *= 2.0 ** -7
    for fmt in FMTS:
        k, kd = to16(x, fmt)
        cache = qsa.alloc_qcache(1, n)
        qsa.qcache_append(k, k, cache, 0)
        want = np.zeros((1, n // 64, oq.REC), dtype=np.uint8)
        oq.append(want, kd, kd, 0, fmt)
        np.testing.assert_array_equal(cache.cpu().numpy(), want)


def test_append_takes_slices_of_a_projection():
    kv, n = 2, 70
    x = torch.randn(n, 12, 128, device="cuda").bfloat16()       # 8 query heads, K, V
    k, v = x[:, 8:10], x[:, 10:]
    a, b = qsa.alloc_qcache(kv, 192), qsa.alloc_qcache(kv, 192)
    qsa.qcache_append(k, v, a, 50)
    qsa.qcache_append(k.contiguous(), v.contiguous(), b, 50)
    assert torch.equal(a, b)
    every = torch.randn(2 * n, kv, 128, device="cuda").half()   # every other token, heads in reverse order of memory
    qsa.qcache_append(every[::2], every[1::2], a, 0)
    qsa.qcache_append(every[::2].contiguous(), every[1::2].contiguous(), b, 0)
    assert torch.equal(a, b)
    ko = torch.zeros(n, 12, 128, device="cuda").half()          # and the reader writes into slices
    qsa.qcache_load(a, ko[:, 2:4], ko[:, 7:9], 0)
    kc, vc = torch.empty(n, kv, 128, device="cuda").half(), torch.empty(n, kv, 128, device="cuda").half()
    qsa.qcache_load(a, kc, vc, 0)
    assert torch.equal(ko[:, 2:4], kc) and torch.equal(ko[:, 7:9], vc)
    assert not ko[:, :2].any() and not ko[:, 4:7].any() and not ko[:, 9:].any()


def test_append_in_pieces_equals_one_call():
    k, _ = to16(_rows(20, 150, 2), oq.BF16)
    v, _ = to16(_rows(21, 150, 2), oq.BF16)
    a, b = qsa.alloc_qcache(2, 256), qsa.alloc_qcache(2, 256)
    qsa.qcache_append(k, v, a, 13)
    at = 0
    for m in (1, 1, 30, 2, 64, 1, 51):
        qsa.qcache_append(k[at:at + m], v[at:at + m], b, 13 + at)
        at += m
    assert at == 150 and torch.equal(a, b)


def test_append_at_a_device_position_in_a_captured_graph():
    """The captured step appends where the device says, replay after replay; positions outside
    the cache are dropped and flagged."""
    k, _ = to16(_rows(30, 5, 2), oq.BF16)
    v, _ = to16(_rows(31, 5, 2), oq.BF16)
    cache, ws = qsa.alloc_qcache(2, 192), _ws()
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qsa.qcache_append(k, v, cache, first, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qsa.qcache_append(k, v, cache, first, ws=ws)
        first += 5
    cache.zero_()
    first.fill_(60)
    want = qsa.alloc_qcache(2, 192)
    for i in range(3):
        graph.replay()
        qsa.qcache_append(k, v, want, 60 + 5 * i)
    assert torch.equal(cache, want) and qsa.read_flags(ws) == 0
    for at, lo, hi in ((189, 0, 3), (-2, 2, 5), (192, 0, 0), (-5, 0, 0), (1 << 30, 0, 0), (-(1 << 30), 0, 0),
                       ((1 << 31) - 1, 0, 0), (-(1 << 31), 0, 0)):
        first.fill_(at)
        graph.replay()
        if hi > lo:
            qsa.qcache_append(k[lo:hi], v[lo:hi], want, at + lo)
        assert torch.equal(cache, want)
        assert qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED


def test_empty_append_and_load_touch_nothing():
    cache = torch.full((1, 1, oq.REC), 9, dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    qsa.qcache_append(none, none, cache, 64)
    qsa.qcache_load(cache, none, none, 64)
    assert (cache == 9).all()


# ------------------------------------------------------------------ attention

def _attend(q, cache, ids, nt, fmt, weights=True, lse=True, f32=False, ws=None, scale=None):
    nq, heads, _ = q.shape
    out = torch.full(q.shape, float("nan"), dtype=torch.float32 if f32 else DT[fmt], device="cuda")
    ls = torch.full((nq, heads), float("nan"), device="cuda") if lse else None
    w = torch.full((nq, cache.shape[0], ids.shape[1]), float("nan"), device="cuda") if weights else None
    d_ids = ids if isinstance(ids, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(ids)).cuda()
    d_nt = nt if isinstance(nt, torch.Tensor) else torch.from_numpy(np.asarray(nt, dtype=np.int32)).cuda()
    qsa.select_attention_qcache(q, cache, d_ids, d_nt, out, ls, w, scale=scale, ws=ws)
    return [None if t is None else t.double().cpu().numpy() for t in (out, ls, w)]


CASES = [
    # nq, kv, group, blocks, tokens (None: ragged), k, valid (None: k)
    (1, 1, 16, 1, 1, 1, None),            # one token
    (1, 1, 1, 2, 65, 2, None),            # one head, a tail block of one token
    (2, 1, 16, 3, 129, 3, None),          # an odd number of blocks
    (3, 2, 8, 40, 2560, 32, None),
    (5, 3, 7, 33, None, 17, None),
    (1, 4, 16, 70, 4477, 64, None),       # one query, the largest selection
    (9, 2, 16, 70, None, 64, "random"),
    (16, 1, 4, 24, None, 7, "random"),    # rows that select nothing among them
    (80, 4, 16, 48, None, 32, None),      # more units than fit at once
    (61, 8, 5, 20, None, 17, "random"),
    (200, 4, 16, 12, None, 4, None),
    (90, 4, 16, 70, None, 64, "random"),  # the largest selections, several units per CTA
    (160, 2, 8, 70, 4477, 64, None),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", CASES, ids=[f"nq{c[0]}-kv{c[1]}x{c[2]}-k{c[5]}" for c in CASES])
def test_attention_matches_the_oracle(case, fmt):
    nq, kv, group, blocks, tokens, k, valid = case
    rng = np.random.default_rng(nq * 100 + k)
    nt = np.full(nq, tokens) if tokens else rng.integers(1, blocks * 64 + 1, size=nq)
    if valid == "random":
        valid = rng.integers(0, k + 1, size=nq)
        valid[nq // 2] = 0
    ids = random_ids(nq + k, nq, k, nt, valid)
    host = random_cache(nq + blocks, kv, blocks, fmt)
    cache = torch.from_numpy(host).cuda()
    q, qd = to16(rng.normal(size=(nq, kv * group, 128)) * 1.5, fmt)
    scale = float(np.float32(128 ** -0.5))
    want = oq.attention(qd, host, ids, nt, scale, fmt)
    ws = _ws()
    check_attention(_attend(q, cache, ids, nt, fmt, ws=ws), want, fmt)
    check_attention(_attend(q, cache, ids, nt, fmt, f32=True, ws=ws), want, fmt, out_f32=True)
    assert qsa.read_flags(ws) == 0
    none = (ids < 0).all(1)
    got = _attend(q, cache, ids, nt, fmt)
    assert not got[0][none].any() and np.isneginf(got[1][none]).all() and not got[2][none].any()


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_same_values_with_and_without_the_optional_outputs(fmt):
    host = random_cache(1, 2, 20, fmt)
    cache = torch.from_numpy(host).cuda()
    q, _ = to16(np.random.default_rng(2).normal(size=(7, 32, 128)), fmt)
    nt = np.full(7, 1280)
    ids = random_ids(3, 7, 12, nt)
    full = _attend(q, cache, ids, nt, fmt, ws=_ws())
    for w in (True, False):
        for l in (True, False):
            got = _attend(q, cache, ids, nt, fmt, weights=w, lse=l)
            np.testing.assert_array_equal(got[0], full[0])
            for a, b in zip(got[1:], full[1:]):
                assert a is None or np.array_equal(a, b)
    again = _attend(q, cache, ids, nt, fmt)
    for a, b in zip(again, full):
        np.testing.assert_array_equal(a, b)   # run to run


def test_attention_takes_slices_of_a_projection():
    fmt = oq.BF16
    cache = torch.from_numpy(random_cache(4, 2, 10, fmt)).cuda()
    x, _ = to16(np.random.default_rng(5).normal(size=(6, 40, 128)), fmt)
    nt = np.full(6, 640)
    ids = random_ids(6, 6, 5, nt)
    for view in (x[:, 4:36], x[:, :32].flip(0).flip(0), x[::2, 8:24], x.transpose(0, 1)[:6, :4]):
        got = _attend(view, cache, ids[:view.shape[0]], nt[:view.shape[0]], fmt)
        want = _attend(view.contiguous(), cache, ids[:view.shape[0]], nt[:view.shape[0]], fmt)
        for a, b in zip(got, want):
            np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_unsorted_repeated_and_bad_ids(fmt):
    rng = np.random.default_rng(7)
    nq, kv, k, blocks = 6, 2, 24, 30
    nt = rng.integers(700, blocks * 64 + 1, size=nq)
    ids = random_ids(8, nq, k, nt, np.full(nq, 10))
    for i in range(nq):
        nb = (nt[i] + 63) // 64
        row = ids[i]
        row[10:15] = [row[0], row[0], nb, blocks + 3, -9]       # repeats, past the context, past the cache, negative
        if i == 0:
            row[15] = np.iinfo(np.int32).max
        ids[i] = rng.permutation(row)
    host = random_cache(9, kv, blocks, fmt)
    q, qd = to16(rng.normal(size=(nq, kv * 16, 128)), fmt)
    ws = _ws()
    got = _attend(q, torch.from_numpy(host).cuda(), ids, nt, fmt, ws=ws)
    check_attention(got, oq.attention(qd, host, ids, nt, float(np.float32(128 ** -0.5)), fmt), fmt)
    assert qsa.read_flags(ws) == qsa.FLAG_BAD_ID


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_ignores_what_lies_past_the_context(fmt):
    """Codes and pairs of every token past the context filled with ones (NaN pairs): the same bits."""
    nq, kv, blocks = 4, 2, 12
    nt = np.array([1, 70, 511, 768 - 37])
    host = random_cache(10, kv, blocks, fmt)
    ids = random_ids(11, nq, 6, nt)
    q, _ = to16(np.random.default_rng(12).normal(size=(nq, kv * 16, 128)), fmt)
    want = _attend(q, torch.from_numpy(host).cuda(), ids, nt, fmt)
    for i in range(nq):
        bad = host.copy()
        for g in range(kv):
            for t in range(int(nt[i]), blocks * 64):
                oq.write_token(bad, g, t, "k", np.full(128, 15), np.nan, np.nan, fmt)
                oq.write_token(bad, g, t, "v", np.full(128, 15), np.nan, np.nan, fmt)
        got = _attend(q[i:i + 1], torch.from_numpy(bad).cuda(), ids[i:i + 1], nt[i:i + 1], fmt)
        clean = _attend(q[i:i + 1], torch.from_numpy(host).cuda(), ids[i:i + 1], nt[i:i + 1], fmt)
        for a, b, c in zip(got, clean, want):
            np.testing.assert_array_equal(a, b)
            assert np.isfinite(a).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_clamps_the_context(fmt):
    host = random_cache(13, 1, 6, fmt)
    cache = torch.from_numpy(host).cuda()
    q, _ = to16(np.random.default_rng(14).normal(size=(3, 16, 128)), fmt)
    ids = np.array([[0, 3, 5], [1, 2, 5], [-1, -1, -1]], dtype=np.int32)
    ws = _ws()
    got = _attend(q, cache, ids, [385, 1 << 30, -4], fmt, ws=ws)
    assert qsa.read_flags(ws) == qsa.FLAG_NBLOCKS_CLAMPED
    want = _attend(q, cache, ids, [384, 384, 0], fmt, ws=ws)
    assert qsa.read_flags(ws) == 0
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)


def _special(seed, fmt, kind):
    """(K, V rows, q) of one KV head whose logits or scales move in an unusual way over the blocks."""
    rng = np.random.default_rng(seed)
    n = 20 * 64
    k, v, q = rng.normal(size=(n, 1, 128)), rng.normal(size=(n, 1, 128)), rng.normal(size=(2, 16, 128))
    t = np.arange(n)[:, None, None]
    if kind == "rising":            # the running maximum grows in every block
        k = k * 0.2 + q[0, 3] * (t // 64) * 0.4
    elif kind == "falling":
        k = k * 0.2 + q[0, 3] * (20 - t // 64) * 0.4
    elif kind == "one":             # one token takes all the weight
        k[777] = 4 * q[0, 5]
    elif kind == "v growing":       # V's scale grows by 2^20 over the blocks
        v = v * np.exp2((t // 64 - 10.0) if fmt == oq.BF16 else (t // 64) * 0.5 - 5)
    elif kind == "v mixed":
        v = v * np.exp2(rng.integers(-8, 9, size=(n, 1, 1)).astype(float))
    elif kind == "v constant":      # scale 0: every row's values are its minimum
        v = np.broadcast_to(rng.normal(size=(n, 1, 1)), v.shape).copy()
    elif kind == "k constant":
        k = np.broadcast_to(rng.normal(size=(n, 1, 1)), k.shape).copy()
    elif kind == "zero queries":
        q[:, ::2] = 0
    elif kind == "unlike heads":    # query heads of very different sizes
        q = q * np.exp2(np.arange(16) - 12.0)[None, :, None]
    elif kind == "unlike dims":     # each head's dimensions over 2^12
        q = q * np.exp2(-(np.arange(128) % 13))[None, None]
    elif kind == "v offset":
        v = v * 0.05 + 30
    elif kind == "flat":            # equal logits
        k = np.zeros_like(k) + rng.normal(size=128)
    return k, v, q


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", ["rising", "falling", "one", "v growing", "v mixed", "v constant", "k constant",
                                  "zero queries", "unlike heads", "unlike dims", "v offset", "flat"])
def test_attention_on_unusual_values(kind, fmt):
    k, v, q = _special(40, fmt, kind)
    n = k.shape[0] - 13
    kt, kd = to16(k[:n], fmt)
    vt, vd = to16(v[:n], fmt)
    cache = qsa.alloc_qcache(1, 20 * 64)
    qsa.qcache_append(kt, vt, cache, 0)
    host = cache.cpu().numpy()
    qt, qd = to16(q, fmt)
    nt = np.array([n, n - 100])
    for kk in (3, 19):
        ids = np.stack([np.sort(np.random.default_rng(kk).permutation(18)[:kk])] * 2).astype(np.int32)
        ids[0, -1] = 19
        want = oq.attention(qd, host, ids, nt, float(np.float32(128 ** -0.5)), fmt)
        check_attention(_attend(qt, cache, ids, nt, fmt), want, fmt)
        check_attention(_attend(qt, cache, ids, nt, fmt, f32=True), want, fmt, out_f32=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [5, 8, 16])
@pytest.mark.parametrize("nq", [3, 160])
@pytest.mark.parametrize("kind", ["rising", "v growing", "one"])
def test_attention_on_unusual_values_in_units_of_many_steps(kind, nq, group, fmt):
    """Units split over a cluster, and so many that each is one CTA's, whose running maxima move in its later steps, too."""
    n = 20 * 64 - 13
    k, v, q = _special(40, fmt, kind)
    kt, _ = to16(k[:n], fmt)
    vt, _ = to16(v[:n], fmt)
    cache = qsa.alloc_qcache(1, 20 * 64)
    qsa.qcache_append(kt, vt, cache, 0)
    qt, qd = to16(np.concatenate([q[:1], q[:1] * 0.5, q[1:]])[np.arange(nq) % 3][:, :group], fmt)
    ids = np.repeat(np.arange(20, dtype=np.int32)[None], nq, 0)
    nt = n - np.arange(nq) // 3
    want = oq.attention(qd, cache.cpu().numpy(), ids, nt, float(np.float32(128 ** -0.5)), fmt)
    check_attention(_attend(qt, cache, ids, nt, fmt), want, fmt)
    check_attention(_attend(qt, cache, ids, nt, fmt, f32=True), want, fmt, out_f32=True)


def test_attention_fp16_lse_has_no_common_shift():
    """What three e4m3 terms leave of a query is at most 2^-10 of 128..256 in the few dimensions below 2^-7 of the
    largest one: 4 of 128 and 2^-10 / sqrt(3) each.  Times the codes' mean, 7.5, it shifts every logit of a head alike:
    1e-3 * 7.5 * scale * (K scale, 0.35) / (128 / 3) = 6e-6, 1.5e-6 of an lse of 4.  With the mean taken back there
    remain the codes' deviations (2.8, and 1 / sqrt(64) of it over a block's tokens): 0.1e-6, beside fp32 sums."""
    fmt, nq = oq.F16, 64
    rng = np.random.default_rng(50)
    kt, _ = to16(rng.normal(size=(640, 2, 128)), fmt)
    vt, _ = to16(rng.normal(size=(640, 2, 128)), fmt)
    cache = qsa.alloc_qcache(2, 640)
    qsa.qcache_append(kt, vt, cache, 0)
    q, qd = to16(rng.normal(size=(nq, 16, 128)), fmt)
    ids = rng.integers(0, 10, size=(nq, 1)).astype(np.int32)
    nt = np.full(nq, 640)
    want = oq.attention(qd, cache.cpu().numpy(), ids, nt, float(np.float32(128 ** -0.5)), fmt)[1]
    got = _attend(q, cache, ids, nt, fmt)[1]
    assert np.linalg.norm(got - want) <= 0.6e-6 * np.linalg.norm(want)


def test_attention_other_scales():
    fmt = oq.BF16
    host = random_cache(15, 1, 9, fmt)
    q, qd = to16(np.random.default_rng(16).normal(size=(2, 16, 128)), fmt)
    nt = np.full(2, 570)
    ids = random_ids(17, 2, 9, nt)
    for scale in (1e-3, 0.5, 2.0):
        s = float(np.float32(scale))
        check_attention(_attend(q, torch.from_numpy(host).cuda(), ids, nt, fmt, scale=s),
                        oq.attention(qd, host, ids, nt, s, fmt), fmt)


def test_attention_nan_rows_and_queries_reach_only_their_own_outputs():
    fmt = oq.BF16
    k, v, q = _special(41, fmt, "plain")
    k[100, 0, 5], v[500, 0, 7], q[1, 4, 0] = np.nan, np.inf, np.inf
    kt, _ = to16(k, fmt)
    vt, _ = to16(v, fmt)
    qt, _ = to16(q, fmt)
    cache = qsa.alloc_qcache(1, 20 * 64)
    qsa.qcache_append(kt, vt, cache, 0)
    out, lse, w = _attend(qt, cache, np.array([[0, 2, 3], [4, 5, 6]], dtype=np.int32), [1280, 1280], fmt)
    assert np.isfinite(out[0]).all() and np.isfinite(lse[0]).all() and np.isfinite(w[0]).all()
    heads = np.arange(16) != 4
    assert np.isnan(out[1, 4]).all() and np.isfinite(out[1, heads]).all() and np.isfinite(lse[1, heads]).all()
    out, lse, w = _attend(qt, cache, np.array([[0, 1, 3], [4, 5, 7]], dtype=np.int32), [1280, 1280], fmt)
    assert np.isnan(out[0]).all() and np.isnan(lse[0]).all()           # block 1 holds the NaN key
    assert np.isnan(out[1, heads]).all() and np.isfinite(lse[1, heads]).all()   # block 7 the infinite value


def test_attention_past_four_gigabytes():
    """Records at offsets past 2^32 bytes, written and attended over where they lie."""
    fmt = oq.BF16
    blocks = 300_000
    cache = qsa.alloc_qcache(2, 64 * blocks)
    assert cache.numel() > 1 << 32
    at = [7, 246_000, 299_999]
    for i, b in enumerate(at):
        k, _ = to16(_rows(50 + i, 64, 2), fmt)
        v, _ = to16(_rows(60 + i, 64, 2), fmt)
        qsa.qcache_append(k, v, cache, 64 * b)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        qsa.qcache_load(cache, ko, vo, 64 * b)
        assert float((ko - k).abs().max()) < 2.0
    small = cache[:, at].contiguous()
    q, qd = to16(np.random.default_rng(18).normal(size=(2, 32, 128)), fmt)
    ids = np.array([at, at], dtype=np.int32)
    got = _attend(q, cache, ids, [64 * blocks, 64 * blocks - 5], fmt)
    near = np.array([[0, 1, 2]] * 2, dtype=np.int32)
    want = _attend(q, small, near, [192, 187], fmt)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)
    check_attention(got, oq.attention(qd, small.cpu().numpy(), near, np.array([192, 187]), float(np.float32(128 ** -0.5)), fmt),
                    fmt)


def test_attention_on_a_side_stream_and_in_a_graph():
    fmt = oq.F16
    host = random_cache(19, 4, 40, fmt)
    cache = torch.from_numpy(host).cuda()
    q, _ = to16(np.random.default_rng(20).normal(size=(3, 64, 128)), fmt)
    nt = np.full(3, 2500)
    ids = random_ids(21, 3, 32, nt)
    want = _attend(q, cache, ids, nt, fmt)
    side = torch.cuda.Stream()
    d_ids, d_nt = torch.from_numpy(ids).cuda(), torch.from_numpy(nt.astype(np.int32)).cuda()
    out, lse = torch.empty_like(q), torch.empty(3, 64, device="cuda")
    w = torch.empty(3, 4, 32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        qsa.select_attention_qcache(q, cache, d_ids, d_nt, out, lse, w)
    side.synchronize()
    np.testing.assert_array_equal(out.double().cpu().numpy(), want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qsa.select_attention_qcache(q, cache, d_ids, d_nt, out, lse, w)
    for seed in (22, 23):
        nq, _ = to16(np.random.default_rng(seed).normal(size=(3, 64, 128)), fmt)
        q.copy_(nq)
        out.zero_()
        graph.replay()
        for a, b in zip((out, lse, w), _attend(q, cache, ids, nt, fmt)):
            np.testing.assert_array_equal(a.double().cpu().numpy(), b)


def test_two_streams_at_once():
    """Calls without a workspace share nothing: two streams, interleaved, each its own result."""
    fmt = oq.BF16
    cache = torch.from_numpy(random_cache(24, 4, 60, fmt)).cuda()
    nt = torch.full((40,), 3840, dtype=torch.int32, device="cuda")
    sets = []
    for seed in (25, 26):
        q, _ = to16(np.random.default_rng(seed).normal(size=(40, 64, 128)), fmt)
        ids = torch.from_numpy(random_ids(seed, 40, 32, np.full(40, 3840))).cuda()
        sets.append((q, ids, _attend(q, cache, ids, nt, fmt)))
    outs = [[(torch.empty_like(q), torch.empty(40, 64, device="cuda"), torch.empty(40, 4, 32, device="cuda"))
             for _ in range(6)] for q, _, _ in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(6):
        for s, (q, ids, _), o in zip(streams, sets, outs):
            with torch.cuda.stream(s):
                qsa.select_attention_qcache(q, cache, ids, nt, *o[i])
    torch.cuda.synchronize()
    for (_, _, want), o in zip(sets, outs):
        for got in o:
            for a, b in zip(got, want):
                np.testing.assert_array_equal(a.double().cpu().numpy(), b)


@pytest.mark.parametrize("fmt", FMTS)
def test_appends_on_two_streams_share_a_block(fmt):
    """Two streams fill one block's tokens in turn, token by token (tokens r and r + 32 share V's bytes): every
    position holds its own row, whatever the streams' order."""
    kv, n = 3, 64
    k, _ = to16(_rows(70, n, kv), fmt)
    v, _ = to16(_rows(71, n, kv), fmt)
    want = qsa.alloc_qcache(kv, 64)
    qsa.qcache_append(k, v, want, 0)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for split in (lambda t: t >= 32, lambda t: t % 2, lambda t: (t // 4) % 2):
        cache = torch.randint(0, 256, tuple(want.shape), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for t in range(32):
            for u in (t, t + 32):
                with torch.cuda.stream(streams[int(split(u))]):
                    qsa.qcache_append(k[u:u + 1], v[u:u + 1], cache, u)
        torch.cuda.synchronize()
        assert torch.equal(cache, want)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_near_the_largest_value_read_as_finite(fmt):
    """The scale is rounded up, so the top level may lie past the format: it reads as the largest finite value, and every
    value within scale / 2 and a rounding of its own."""
    rng = np.random.default_rng(72)
    big = float(torch.finfo(DT[fmt]).max)
    rows = [np.where(rng.random(128) < 0.5, big, 0.0), rng.uniform(0, 1, 128) * big, np.where(np.arange(128) == 3, big, -big / 512),
            np.where(rng.random(128) < 0.5, -big, 0.0), np.full(128, big), np.full(128, -big),
            np.where(np.arange(128) % 2, np.inf, big)]
    rows[1][5] = big
    if fmt == oq.F16:   # a range that fp32 holds
        rows += [np.where(rng.random(128) < 0.5, -big, big), rng.uniform(-1, 1, 128) * big]
        rows[-1][:2] = -big, big
    k, kd = to16(np.stack(rows)[:, None], fmt)
    cache = qsa.alloc_qcache(1, 64)
    qsa.qcache_append(k, k.flip(0), cache, 0)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    qsa.qcache_load(cache, ko, vo, 0)
    with np.errstate(invalid="ignore"):
        _, scale, _ = oq.quantise(kd, fmt)
        want = np.minimum(oq.rows(cache.cpu().numpy(), 0, len(rows), fmt)[0], big)   # NaN stays NaN
    assert np.isnan(want[6]).all() and torch.isnan(ko[6]).all() and torch.isnan(vo[-7]).all()
    ok = np.arange(len(rows)) != 6
    got = ko.double().cpu().numpy()
    np.testing.assert_array_equal(got[ok], torch.from_numpy(want[ok]).to(DT[fmt]).double().numpy())
    assert np.isfinite(got[ok]).all()
    half = float(torch.finfo(DT[fmt]).eps) / 2
    assert (np.abs(got - kd)[ok] <= (scale[..., None] / 2 * (1 + 1e-12) + half * np.abs(got))[ok]).all()
    assert torch.equal(vo.flip(0)[ok.tolist()], ko[ok.tolist()])


@pytest.mark.parametrize("nq", [2, 100])
def test_attention_over_the_largest_values_is_finite(nq):
    """fp16 rows of +-65504: their top level is 65536, which the fp32 output shows and the fp16 output holds at 65504."""
    fmt = oq.F16
    sign = np.where(np.arange(128) % 2, 1.0, -1.0)
    kt, _ = to16(np.random.default_rng(73).normal(size=(300, 1, 128)), fmt)
    vt, _ = to16(np.broadcast_to(65504.0 * sign, (300, 1, 128)), fmt)
    cache = qsa.alloc_qcache(1, 320)
    qsa.qcache_append(kt, vt, cache, 0)
    q, _ = to16(np.random.default_rng(74).normal(size=(nq, 16, 128)), fmt)
    ids = np.repeat(np.arange(5, dtype=np.int32)[None], nq, 0)
    out = _attend(q, cache, ids, np.full(nq, 300), fmt)[0]
    assert (out[..., 1::2] == 65504).all() and (np.abs(out[..., ::2] + 65504) <= 65536 * 2.0 ** -9).all()
    wide = _attend(q, cache, ids, np.full(nq, 300), fmt, f32=True)[0]
    assert (np.abs(wide[..., 1::2] - 65536) <= 65536 * 2.0 ** -9).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_strides_that_no_element_uses(fmt):
    """One token, one query or one head: its stride is never used, whatever torch has it at."""
    x, _ = to16(np.random.default_rng(75).normal(size=(3, 16 * 128 + 4)), fmt)   # rows of a projection, no multiple of 8 long
    row = x[:1].as_strided((1, 16, 128), (x.stride(0), 128, 1))
    assert row.stride(0) % 8 == 4
    a, b = qsa.alloc_qcache(2, 64), qsa.alloc_qcache(2, 64)
    qsa.qcache_append(row[:, 2:4], row[:, 6:8], a, 9)
    qsa.qcache_append(row[:, 2:4].contiguous(), row[:, 6:8].clone(memory_format=torch.contiguous_format), b, 9)
    assert torch.equal(a, b)
    out, _ = to16(np.zeros((1, 4 * 128 + 4)), fmt)
    ko, vo = out.as_strided((1, 2, 128), (516, 128, 1)), out.as_strided((1, 2, 128), (516, 128, 1), 256)
    qsa.qcache_load(a, ko, vo, 9)
    kc, vc = torch.empty(1, 2, 128, dtype=DT[fmt], device="cuda"), torch.empty(1, 2, 128, dtype=DT[fmt], device="cuda")
    qsa.qcache_load(a, kc, vc, 9)
    assert torch.equal(ko, kc) and torch.equal(vo, vc) and not out[:, 512:].any()
    cache = torch.from_numpy(random_cache(76, 1, 4, fmt)).cuda()
    ids = np.array([[0, 2, 3]], dtype=np.int32)
    for view in (row[:, :5], row[:, 3:4], x.as_strided((3, 1, 128), (128, 129, 1))):   # one query; one head of one; one head of three
        n = view.shape[0]
        want = _attend(view.clone(memory_format=torch.contiguous_format), cache, ids.repeat(n, 0), [250] * n, fmt)
        for got, ref in zip(_attend(view, cache, ids.repeat(n, 0), [250] * n, fmt), want):
            np.testing.assert_array_equal(got, ref)
    one = x.as_strided((3, 1, 128), (128, 129, 1))
    c, d = qsa.alloc_qcache(1, 64), qsa.alloc_qcache(1, 64)
    qsa.qcache_append(one, one, c, 5)
    qsa.qcache_append(one.clone(memory_format=torch.contiguous_format), one.clone(memory_format=torch.contiguous_format), d, 5)
    assert torch.equal(c, d)


def test_current_stream_is_the_public_one():
    side = torch.cuda.Stream()
    for s in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(s):
            assert qsa._current_stream(torch.cuda.current_device()) == s.cuda_stream


def _coherent(kind, nq, group):
    """(K, V, q) whose P.V weights round alike over thousands of tokens, so that what the rounding leaves adds up.

    K rows are constant (scale 0), so a block's tokens have one logit, u[block] times the head's factor: 0, or 0.25 in
    every fourth block, which sets the reference.  A head's factor makes 2^y of the others, relative to that, an odd
    number of 1024ths in 0.70 .. 0.80: 10 significant bits, which a weight's fp16 form holds and two e4m3 terms (8 bits)
    do not.  V rows lie between -0.9375 and 0.9375 (scale 1/8 exactly) with 126 dimensions near 0, so at codes 7 and 8.
    rising: the last block's logit moves the references late (by 5 to 8 powers of two); v growing: its scale does (2^5)."""
    rng = np.random.default_rng(60)
    block = np.arange(64 * 64 - 13) // 64
    u, a = np.where(np.arange(64) % 4 == 0, 0.25, 0.0), np.ones(64)
    if kind == "rising":
        u[63] = 4.25
    elif kind == "v growing":
        a[63] = 32
    v = rng.uniform(-0.02, 0.02, (len(block), 128))
    v[:, 0], v[:, 1] = -0.9375, 0.9375
    p = (2 * rng.integers(359, 410, size=(nq, group)) + 1) / 1024
    rest = -np.log(p) * 128 ** 0.5 / 0.25
    hold = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().double().numpy()  # noqa: E731
    q = hold(rng.normal(size=(nq, group, 128)) * 0.05)
    q[..., :4] = 0
    rest -= q.sum(-1)
    for i in range(4):                                  # the sum to 32 bits
        q[..., i] = hold(rest)
        rest -= q[..., i]
    return np.repeat(u[block][:, None, None], 128, 2), (v * a[block][:, None])[:, None], q


@pytest.mark.parametrize("group", [5, 16])
@pytest.mark.parametrize("nq", [3, 80])
@pytest.mark.parametrize("kind", ["even", "rising", "v growing"])
def test_attention_returns_what_the_weights_rounding_leaves(kind, nq, group):
    """bf16, split over a cluster (3 queries) and not (80), half groups and whole ones.  What the rounding leaves of a weight w,
    at most 2^-8 of it, is returned at the mean code, 7.5, so a code c keeps 2^-8 w |c - 7.5|; the codes of a
    dimension are 7 or 8 at random, so those add up as a random walk: 1.5 of its deviation bounds the norm over 126
    dimensions.  To that the fp32 arithmetic: 128 additions of a product (2^-17) at most truncated (2^-16), a logit
    below 16 (2^-20) and its power, 40 additions of the sum of weights (2^-18.7): 2^-15 of the sum of magnitudes
    in all.  Without the return the error is 3 ("rising") to 11 times this bound by the same arithmetic, with
    what is left not moved along with the references hundreds of times."""
    fmt = oq.BF16
    k, v, q = _coherent(kind, nq, group)
    n = len(k)
    kt, _ = to16(k, fmt)
    vt, _ = to16(v, fmt)
    qt, qd = to16(q, fmt)
    cache = qsa.alloc_qcache(1, 64 * 64)
    qsa.qcache_append(kt, vt, cache, 0)
    chosen = np.r_[0:60, 63]
    ids = np.repeat(chosen.astype(np.int32)[None], nq, 0)
    got = _attend(qt, cache, ids, np.full(nq, n), fmt, f32=True)[0]
    host = cache.cpu().numpy()
    codes, pairs = zip(*(oq.read_block(host[0, b], fmt)[1:] for b in chosen))
    seen = (64 * chosen[:, None] + np.arange(64) < n).reshape(-1)
    codes = np.concatenate(codes)[seen]
    ks, km, vs, vm = (np.concatenate([x[w, :, j] for x in pairs])[seen] for w in (0, 1) for j in (0, 1))
    assert not ks.any() and (np.abs(codes[:, 2:] - 7.5) == 0.5).all()
    s = float(np.float32(128 ** -0.5)) * qd.sum(-1)[..., None] * km
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    w = p * vs
    want = w @ codes + (p @ vm)[..., None]
    bound = 1.5 * 2.0 ** -8 * np.sqrt(w ** 2 @ (codes - 7.5) ** 2) + 2.0 ** -15 * (w @ codes + (p @ np.abs(vm))[..., None])
    assert np.linalg.norm((got - want)[..., 2:]) <= np.linalg.norm(bound[..., 2:])


@pytest.mark.parametrize("fmt", FMTS)
def test_head_major_views(fmt):
    """Rows kept head by head in memory: the append, the reader and the attention take them as they lie."""
    kv, n = 3, 70
    x, _ = to16(_rows(77, kv, n), fmt)                     # [kv, n, 128] in memory
    y, _ = to16(_rows(78, kv, 2 * n), fmt)
    k, v = x.transpose(0, 1), y[:, ::2].transpose(0, 1)    # [n, kv, 128]
    assert not k.is_contiguous() and k.stride(1) > k.stride(0)
    a, b = qsa.alloc_qcache(kv, 128), qsa.alloc_qcache(kv, 128)
    qsa.qcache_append(k, v, a, 31)
    qsa.qcache_append(k.contiguous(), v.contiguous(), b, 31)
    assert torch.equal(a, b)
    ko, vo = torch.zeros_like(x), torch.zeros_like(y)
    qsa.qcache_load(a, ko.transpose(0, 1), vo[:, ::2].transpose(0, 1), 31)
    kc, vc = torch.empty(n, kv, 128, dtype=DT[fmt], device="cuda"), torch.empty(n, kv, 128, dtype=DT[fmt], device="cuda")
    qsa.qcache_load(a, kc, vc, 31)
    assert torch.equal(ko.transpose(0, 1), kc) and torch.equal(vo[:, ::2].transpose(0, 1), vc) and not vo[:, 1::2].any()
    cache = torch.from_numpy(random_cache(79, 2, 10, fmt)).cuda()
    heads, _ = to16(np.random.default_rng(80).normal(size=(32, 6, 128)), fmt)   # [heads, nq, 128] in memory
    nt = np.full(6, 640)
    ids = random_ids(81, 6, 5, nt)
    view = heads.transpose(0, 1)
    for got, ref in zip(_attend(view, cache, ids, nt, fmt), _attend(view.contiguous(), cache, ids, nt, fmt)):
        np.testing.assert_array_equal(got, ref)
