"""The 4-bit cache and the eviction on the CPU: pins of the oracle, and the argument checks of
the library and of the binding (no kernel runs)."""
import numpy as np
import pytest

from oracle import qcache as oq
from sparse_attention_kv_gb300 import _build, qsa

FAKE = 1 << 20
FAR = 1 << 34   # a second range that overlaps no other

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return qsa.load()


# ------------------------------------------------------------------ oracle pins

@pytest.mark.parametrize("fmt", [oq.BF16, oq.F16])
def test_round_up_is_the_next_value_of_the_format(fmt):
    bits = np.arange(1, 0x7C00 if fmt == oq.F16 else 0x7F80, 37, dtype=np.uint16)
    v = oq.bits_to_f64(bits, fmt)
    np.testing.assert_array_equal(oq.round_up(v, fmt), v)                      # held values stay
    below = oq.bits_to_f64(bits - 1, fmt)
    np.testing.assert_array_equal(oq.round_up(below + (v - below) * 2.0 ** -12, fmt), v)


def test_quantise_by_hand():
    x = np.zeros((1, 128))
    x[0, :4] = [-1.0, 14.0, 0.5, 1.5]        # range 15: scale 1, ties at 1.5 and 2.5
    c, s, lo = oq.quantise(x, oq.BF16)
    assert s[0] == 1.0 and lo[0] == -1.0
    assert c[0, :5].tolist() == [0, 15, 2, 2, 1]
    c, s, lo = oq.quantise(np.full((1, 128), 3.25), oq.F16)                     # a constant row
    assert s[0] == 0.0 and lo[0] == 3.25 and not c.any()
    for bad in (np.inf, -np.inf, np.nan):
        x[0, 7] = bad
        c, s, lo = oq.quantise(x, oq.BF16)
        assert np.isnan(s[0]) and np.isnan(lo[0]) and not c.any()


@pytest.mark.parametrize("fmt", [oq.BF16, oq.F16])
def test_values_are_within_half_a_step(fmt):
    rng = np.random.default_rng(3)
    x = oq.bits_to_f64(oq.f64_to_bits(rng.normal(size=(200, 128)).astype(np.float32), fmt), fmt)
    c, s, lo = oq.quantise(x, fmt)
    assert (np.abs(s[:, None] * c + lo[:, None] - x) <= s[:, None] / 2 * (1 + 1e-12)).all()
    assert c.max() == 15 and c.min() == 0


def test_record_layout_round_trip():
    rng = np.random.default_rng(4)
    cache = np.zeros((2, 2, oq.REC), dtype=np.uint8)
    k, v = (oq.bits_to_f64(oq.f64_to_bits(rng.normal(size=(100, 2, 128)).astype(np.float32), oq.BF16), oq.BF16)
            for _ in range(2))
    oq.append(cache, k, v, 20, oq.BF16)
    kb, vb = oq.rows(cache, 20, 100, oq.BF16)
    for got, x in ((kb, k), (vb, v)):
        c, s, lo = oq.quantise(x, oq.BF16)
        np.testing.assert_array_equal(got, s[..., None] * c + lo[..., None])
    # one dimension of one token, byte by byte
    c, _, _ = oq.quantise(v, oq.BF16)
    t, d = 45, 77                                   # token 45 of block 0: plane 0, byte 13, high nibble
    assert cache[1, 0, oq.VCODE + d * 16 + 13] >> 4 == c[t - 20, 1, d]
    ck, _, _ = oq.quantise(k, oq.BF16)
    assert cache[0, 0, 0 * 1024 + t * 16 + 13] >> 4 == ck[t - 20, 0, 77]   # dimension 64 + 13


def test_plan_by_hand():
    w = np.array([0, 5, 1, np.nan, 5, 2, 0, 0], dtype=np.float32)
    kept, left = oq.evict_plan(w, 8 * 64 - 3, 4, 1, 1)
    assert kept.tolist() == [0, 1, 4, 7] and left == 4 * 64 - 3
    kept, left = oq.evict_plan(w, 8 * 64, 3, 0, 1)
    assert kept.tolist() == [1, 4, 7]
    kept, left = oq.evict_plan(w, 100, 4, 1, 1)
    assert kept.tolist() == [0, 1, -1, -1] and left == 100
    kept, _ = oq.evict_plan(np.zeros(6, np.float32), 6 * 64, 3, 0, 1)          # ties to the lower id
    assert kept.tolist() == [0, 1, 5]


# ------------------------------------------------------------------ refusals of the library

def test_cache_bytes(lib):
    assert lib.qsa_qcache_bytes(4, 8192) == 4 * 128 * qsa.QCACHE_BLOCK_BYTES
    assert lib.qsa_qcache_bytes(2, 1 << 30) == 2 * (1 << 24) * qsa.QCACHE_BLOCK_BYTES
    for bad in ((0, 64), (65536, 64), (1, 0), (1, 100), (1, -64), (1, (1 << 30) + 64)):
        assert lib.qsa_qcache_bytes(*bad) == 0


ROWS = [
    (dict(k=None), "ARG"), (dict(v=None), "ARG"), (dict(cache=None), "ARG"), (dict(k=FAKE + 8), "ARG"),
    (dict(cache=FAKE + 4), "ARG"), (dict(ks=(12, 128)), "ARG"), (dict(vs=(512, 4)), "ARG"), (dict(n=-1), "ARG"),
    (dict(n=4097), "ARG"), (dict(first=-1), "ARG"), (dict(first=4093), "ARG"), (dict(kv=0), "ARG"),
    (dict(kv=65536), "ARG"), (dict(D=64), "ARG"), (dict(cap=100), "ARG"), (dict(cap=0), "ARG"),
    (dict(cap=(1 << 30) + 64), "ARG"), (dict(dt=qsa.F32), "UNSUPPORTED"), (dict(dt=qsa.E4M3), "UNSUPPORTED"),
]
STATUS = {"ARG": qsa.ERR_INVALID_ARG, "UNSUPPORTED": qsa.ERR_UNSUPPORTED, "WS": qsa.ERR_WORKSPACE, "OK": qsa.OK}


@pytest.mark.parametrize("case,status", ROWS + [
    (dict(ws=FAKE + 64), "WS"), (dict(ws_bytes=128), "WS"), (dict(n=0), "OK"), (dict(n=0, first=4096), "OK"),
    (dict(n=4097, dev=FAKE), "ARG")])
def test_append_rejects_bad_arguments_before_launch(lib, case, status):
    a = dict(k=FAKE, ks=(512, 128), v=FAKE, vs=(512, 128), dt=qsa.BF16, n=4, kv=4, D=128, first=0, dev=None, cache=FAKE,
             cap=4096, ws=FAKE, ws_bytes=256)
    a.update(case)
    st = lib.qsa_qcache_append(a["k"], *a["ks"], a["v"], *a["vs"], a["dt"], a["n"], a["kv"], a["D"], a["first"], a["dev"],
                               a["cache"], a["cap"], a["ws"], a["ws_bytes"], None)
    assert st == STATUS[status]
    assert status == "OK" or lib.qsa_last_error().decode()


@pytest.mark.parametrize("case,status", ROWS + [(dict(n=0), "OK")])
def test_load_rejects_bad_arguments_before_launch(lib, case, status):
    a = dict(k=FAKE, ks=(512, 128), v=FAKE, vs=(512, 128), dt=qsa.BF16, n=4, kv=4, D=128, first=0, cache=FAKE, cap=4096)
    a.update(case)
    st = lib.qsa_qcache_load(a["cache"], a["dt"], a["kv"], a["D"], a["cap"], a["first"], a["n"], a["k"], *a["ks"], a["v"],
                             *a["vs"], None)
    assert st == STATUS[status]


@pytest.mark.parametrize("case,status", [
    (dict(qa=None), "ARG"), (dict(cache=None), "ARG"), (dict(ids=None), "ARG"), (dict(nt=None), "ARG"),
    (dict(out=None), "ARG"), (dict(nq=0), "ARG"), (dict(D=64), "ARG"), (dict(kv=0), "ARG"), (dict(heads=0), "ARG"),
    (dict(heads=63), "ARG"), (dict(heads=68, kv=4), "ARG"), (dict(k=0), "ARG"), (dict(k=65), "ARG"),
    (dict(cap=100), "ARG"), (dict(qs=(100, 128)), "ARG"), (dict(qs=(8192, 4)), "ARG"), (dict(qa=FAKE + 8), "ARG"),
    (dict(out=FAKE + 8), "ARG"), (dict(scale=0.0), "ARG"), (dict(scale=float("nan")), "ARG"),
    (dict(scale=float("inf")), "ARG"), (dict(odt=qsa.F16), "ARG"), (dict(odt=qsa.E4M3), "ARG"),
    (dict(nq=1 << 26, kv=4), "ARG"), (dict(dt=qsa.F32), "UNSUPPORTED"), (dict(ws=FAKE + 64), "WS"),
    (dict(ws_bytes=16), "WS"),
])
def test_attention_rejects_bad_arguments_before_launch(lib, case, status):
    a = dict(qa=FAKE, qs=(8192, 128), dt=qsa.BF16, cache=FAKE, ids=FAKE, k=32, nt=FAKE, nq=4, heads=64, kv=4, D=128,
             cap=4096, scale=0.1, out=FAKE, odt=qsa.BF16, ws=FAKE, ws_bytes=256)
    a.update(case)
    st = lib.qsa_select_attention_qcache(a["qa"], *a["qs"], a["dt"], a["cache"], a["ids"], a["k"], a["nt"], a["nq"],
                                         a["heads"], a["kv"], a["D"], a["cap"], a["scale"], a["out"], a["odt"], None, None,
                                         a["ws"], a["ws_bytes"], None)
    assert st == STATUS[status]
    assert lib.qsa_last_error().decode()


@pytest.mark.parametrize("case,status", [
    (dict(w=None), "ARG"), (dict(ids=None), "ARG"), (dict(acc=None), "ARG"), (dict(nq=0), "ARG"), (dict(kv=0), "ARG"),
    (dict(k=0), "ARG"), (dict(nq=1 << 20), "ARG"), (dict(nq=1 << 30, kv=1 << 30), "ARG"), (dict(n=0), "ARG"),
    (dict(n=(1 << 24) + 1), "ARG"), (dict(decay=-0.5), "ARG"), (dict(decay=float("nan")), "ARG"),
    (dict(decay=float("inf")), "ARG"), (dict(ws=FAKE + 8), "WS"), (dict(ws_bytes=255), "WS"),
    (dict(prev=FAKE + 396), "ARG"), (dict(prev=FAKE - 4), "ARG"),   # overlaps acc without being it
])
def test_weights_add_rejects_bad_arguments_before_launch(lib, case, status):
    a = dict(w=FAKE, ids=FAKE, nq=4, kv=4, k=32, decay=1.0, prev=None, acc=FAKE, n=100, ws=FAKE, ws_bytes=256)
    a.update(case)
    st = lib.qsa_block_weights_add(a["w"], a["ids"], a["nq"], a["kv"], a["k"], a["decay"], a["prev"], a["acc"], a["n"], a["ws"],
                                   a["ws_bytes"], None)
    assert st == STATUS[status]
    assert lib.qsa_last_error().decode()


@pytest.mark.parametrize("case,status", [
    (dict(w=None), "ARG"), (dict(nt=None), "ARG"), (dict(keep=None), "ARG"), (dict(new=None), "ARG"), (dict(rows=0), "ARG"),
    (dict(rows=(1 << 20) + 1), "ARG"), (dict(n=0), "ARG"), (dict(n=(1 << 24) + 1, stride=1 << 25), "ARG"),
    (dict(stride=99), "ARG"), (dict(n_keep=0), "ARG"), (dict(n_keep=101), "ARG"), (dict(first=-1), "ARG"),
    (dict(last=0), "ARG"), (dict(first=40, last=11), "ARG"), (dict(first=(1 << 31) - 1, last=(1 << 31) - 1), "ARG"),
    (dict(ws_bytes=8), "WS"),
])
def test_plan_rejects_bad_arguments_before_launch(lib, case, status):
    a = dict(w=FAKE, stride=100, nt=FAKE, rows=2, n=100, n_keep=50, first=1, last=2, keep=FAKE, new=FAKE, ws=FAKE,
             ws_bytes=256)
    a.update(case)
    st = lib.qsa_evict_plan(a["w"], a["stride"], a["nt"], a["rows"], a["n"], a["n_keep"], a["first"], a["last"], a["keep"],
                            a["new"], a["ws"], a["ws_bytes"], None)
    assert st == STATUS[status]
    assert lib.qsa_last_error().decode()


@pytest.mark.parametrize("arrays,n_keep,status", [
    ([], 4, "ARG"),
    ([(FAKE, FAR, 64, 1, 8, 8)] * 9, 4, "ARG"),
    ([(None, FAR, 64, 1, 8, 8)], 4, "ARG"),
    ([(FAKE, None, 64, 1, 8, 8)], 4, "ARG"),
    ([(FAKE, FAR, 64, 0, 8, 8)], 4, "ARG"),
    ([(FAKE, FAR, 64, 1, 0, 8)], 4, "ARG"),
    ([(FAKE, FAR, 64, 1, 8, 3)], 4, "ARG"),                # fewer destination blocks than kept
    ([(FAKE, FAR, 0, 1, 8, 8)], 4, "ARG"),
    ([(FAKE, FAR, 6, 1, 8, 8)], 4, "ARG"),
    ([(FAKE + 2, FAR, 64, 1, 8, 8)], 4, "ARG"),
    ([(FAKE, FAR + 1, 64, 1, 8, 8)], 4, "ARG"),
    ([(FAKE, FAR, 64, 1, 8, 8)], 0, "ARG"),
    ([(FAKE, FAKE, 64, 1, 8, 8)], 4, "ARG"),               # in place
    ([(FAKE, FAKE + 64 * 7, 64, 1, 8, 8)], 4, "ARG"),      # overlaps its source's last record
    ([(FAKE, FAR, 64, 1, 8, 8), (FAKE, FAR + 64, 64, 1, 8, 8)], 4, "ARG"),           # two destinations
    ([(FAKE, FAR, 64, 1, 8, 8), (FAR + 128, FAR + 4096, 64, 1, 8, 8)], 4, "ARG"),    # another array's source
])
def test_gather_rejects_bad_arguments_before_launch(lib, arrays, n_keep, status):
    packed = (qsa.BlockArray * max(1, len(arrays)))(*(qsa.BlockArray(*a) for a in arrays))
    assert lib.qsa_gather_blocks(packed, len(arrays), FAKE, n_keep, None, 0, None) == STATUS[status]
    assert lib.qsa_last_error().decode()


def test_gather_rejects_null_and_small_workspace(lib):
    one = (qsa.BlockArray * 1)(qsa.BlockArray(FAKE, FAR, 64, 1, 8, 8))
    assert lib.qsa_gather_blocks(None, 1, FAKE, 4, None, 0, None) == qsa.ERR_INVALID_ARG
    assert lib.qsa_gather_blocks(one, 1, None, 4, None, 0, None) == qsa.ERR_INVALID_ARG
    assert lib.qsa_gather_blocks(one, 1, FAKE, 4, FAKE, 100, None) == qsa.ERR_WORKSPACE


# ------------------------------------------------------------------ refusals of the binding

def test_binding_checks_shapes_before_devices(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    rows, cache = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(2, 3, 8704, dtype=torch.uint8)
    for k, v, c, first in ((rows, rows.half(), cache, 0), (rows, rows[:3], cache, 0), (rows.float(), rows.float(), cache, 0),
                           (rows[:, :1], rows[:, :1], cache, 0), (rows, rows, cache[:, :, :100], 0),
                           (rows, rows, cache.int(), 0), (rows[..., ::2], rows[..., ::2], cache, 0),
                           (rows, rows, cache, torch.zeros(2, dtype=torch.int32)), (rows, rows, cache, torch.zeros(1))):
        with pytest.raises(ValueError):
            qsa.qcache_append(k, v, c, first)
    with pytest.raises(ValueError, match="current device"):   # CPU tensors
        qsa.qcache_append(rows, rows, cache, 0)
    with pytest.raises(ValueError, match="current device"):
        qsa.qcache_load(cache, rows, rows)
    ids, nt, out = torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros_like(rows)
    for bad in (dict(ids=ids.long()), dict(ids=ids[:3]), dict(n_tokens=nt.long()), dict(n_tokens=nt[:2]),
                dict(out=out.half()), dict(out=out[:, :1]), dict(lse=torch.zeros(4, 3)), dict(weights=torch.zeros(4, 2, 7)),
                dict(weights=torch.zeros(4, 8, 2).transpose(1, 2))):
        a = dict(ids=ids, n_tokens=nt, out=out)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.select_attention_qcache(rows, cache, **a)
    with pytest.raises(ValueError, match="current device"):
        qsa.select_attention_qcache(rows, cache, ids, nt, out)
    w, acc = torch.zeros(4, 2, 8), torch.zeros(10)
    for bad in (dict(weights=w.double()), dict(ids=ids[:, :7]), dict(acc=acc[::2]), dict(prev=torch.zeros(9))):
        a = dict(weights=w, ids=ids, acc=acc, prev=None)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.block_weights_add(**a)
    keep, one = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for bad in (dict(weights=acc), dict(keep=keep[0]), dict(n_tokens=nt), dict(new_tokens=one.long())):
        a = dict(weights=acc[None], n_tokens=one, keep=keep, new_tokens=one)
        a.update(bad)
        with pytest.raises(ValueError):
            qsa.evict_plan(**a)
    for arrays in ([], [(acc, acc.double())], [(cache, cache[:1])], [(cache, torch.zeros(2, 3, 100, dtype=torch.uint8))],
                   [(cache.transpose(0, 1), cache.transpose(0, 1))]):
        with pytest.raises(ValueError):
            qsa.gather_blocks(arrays, keep[0])


def test_alloc_rejects_bad_sizes(lib):
    with pytest.raises(ValueError):
        qsa.alloc_qcache(1, 100)


@pytest.mark.parametrize("case", [
    dict(new=FAKE + 4), dict(new=FAKE - 4),                # overlaps n_tokens without being it
    dict(keep=FAKE + 4), dict(keep=FAKE - 4 * 99),         # overlaps n_tokens
    dict(new=FAR + 4 * 99), dict(keep=FAR),                # overlaps the weights' second row
    dict(keep=FAR, w=3 * FAR, new=FAR + 4 * 99), dict(keep=FAR + 4 * 199),
])
def test_plan_rejects_overlapping_arrays(lib, case):
    a = dict(w=FAR, nt=FAKE, keep=2 * FAR, new=FAKE)
    a.update(case)
    st = lib.qsa_evict_plan(a["w"], 100, a["nt"], 2, 100, 50, 1, 2, a["keep"], a["new"], None, 0, None)
    assert st == qsa.ERR_INVALID_ARG
    assert "overlap" in lib.qsa_last_error().decode()


def test_decay_crosses_the_boundary_in_64_bits(lib):
    import ctypes
    import os
    import re
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qsa.h")).read()
    declared = re.search(r"qsa_block_weights_add\((.*?)\);", header, flags=re.S).group(1).split(",")
    at = next(i for i, x in enumerate(declared) if x.split()[-1] == "decay")
    assert declared[at].split()[0] == "double" and lib.qsa_block_weights_add.argtypes[at] is ctypes.c_double


@pytest.mark.parametrize("case", [dict(acc=FAKE + 4 * (4 * 4 * 32) - 4), dict(acc=FAKE - 4 * 99), dict(ids=FAR + 4 * 99),
                                  dict(ids=FAR - 4 * (4 * 32 - 1))])
def test_weights_add_rejects_an_acc_that_overlaps_its_inputs(lib, case):
    a = dict(w=FAKE, ids=2 * FAR, acc=FAR)
    a.update(case)
    st = lib.qsa_block_weights_add(a["w"], a["ids"], 4, 4, 32, 1.0, None, a["acc"], 100, None, 0, None)
    assert st == qsa.ERR_INVALID_ARG and "overlap" in lib.qsa_last_error().decode()


@pytest.mark.parametrize("keep", [FAR + 64 * 8 - 4, FAR - 12, FAR + 64])
def test_gather_rejects_a_keep_inside_a_destination(lib, keep):
    one = (qsa.BlockArray * 1)(qsa.BlockArray(FAKE, FAR, 64, 1, 8, 8))
    assert lib.qsa_gather_blocks(one, 1, keep, 4, None, 0, None) == qsa.ERR_INVALID_ARG
    assert "keep" in lib.qsa_last_error().decode()


def test_current_stream_needs_no_internal_name(monkeypatch):
    class Stream:
        cuda_stream = 77
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Stream())
    assert qsa._current_stream(0) == 77
