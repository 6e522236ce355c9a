"""Inputs and bounds shared by the GPU tests of the 4-bit cache and the eviction."""
import numpy as np
import torch

from oracle import qcache as oq

DT = {oq.BF16: torch.bfloat16, oq.F16: torch.float16}


def to16(x, fmt):
    """x (any float array) on the GPU in the 16-bit format, and those values in float64."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DT[fmt])
    return t.cuda(), t.double().numpy()


def random_cache(seed, kv, blocks, fmt):
    """A filled cache (numpy uint8): uniform codes, scales and minima of about normal rows."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, size=(kv, blocks, oq.REC), dtype=np.uint8)
    scale = rng.uniform(0.2, 0.45, size=(kv, blocks, 2, 64))
    low = -scale * rng.uniform(6, 9, size=scale.shape)
    pairs = np.stack([scale, low], axis=-1).astype(np.float32)
    bits = torch.from_numpy(pairs).to(DT[fmt]).view(torch.int16).numpy().view(np.uint16)
    c[:, :, oq.KPAIR:oq.VCODE] = np.ascontiguousarray(bits).view(np.uint8).reshape(kv, blocks, -1)
    return c


def random_ids(seed, nq, k, n_tokens, valid=None):
    """Distinct ascending ids per query inside its context (the last block often among them), -1 behind."""
    rng = np.random.default_rng(seed)
    ids = np.full((nq, k), -1, dtype=np.int32)
    for i in range(nq):
        nb = (int(n_tokens[i]) + 63) // 64
        m = min(nb, k if valid is None else int(valid[i]))
        pick = rng.permutation(nb)[:m]
        if m and rng.random() < 0.7 and nb - 1 not in pick:
            pick[0] = nb - 1
        ids[i, :m] = np.sort(pick)
    return ids


def check_attention(got, want, fmt, out_f32=False):
    """(out, lse, weights) of the library against the oracle's, each within a bound made of the
    roundings: weights of the P.V product held to 2^-8 of themselves beside bf16 rows (two 4-bit
    significands) and 2^-11 beside fp16 ones, and to 2^-17 of the largest weight times the
    largest V scale where they are small; 128 fp32 additions (2^-17 of the sum of magnitudes) in a
    logit, twice that in a weight; 2^-14 for the fp32 sums over the tokens; half a step of the
    output's type."""
    out, lse, weights = got
    ref, ref_lse, ref_w, info = want
    nq, heads, _ = ref.shape
    kv = ref_w.shape[1]
    delta = 2.0 ** -8 if fmt == oq.BF16 else 2.0 ** -11
    half = 2.0 ** -24 if out_f32 else (2.0 ** -8 if fmt == oq.BF16 else 2.0 ** -11)
    eps = 2.0 ** -17 * info["logit"]
    step = np.repeat(info["vstep"], heads // kv, axis=1)
    floor = 2.0 ** -17 * info["top"] * info["tokens"][:, None] * 15 * step
    reach = info["mass"] + info["least"][..., None]
    bound = delta * info["mass"] + floor[..., None] + (2 * eps + 2.0 ** -14)[..., None] * reach + half * np.abs(ref) + \
        (2.0 ** -24 if fmt == oq.F16 else 0.0)
    assert np.isfinite(out).all()
    err = np.abs(out - ref)
    assert (err <= bound).all(), f"out off by {np.max(err / np.maximum(bound, 1e-30)):.3g} x its bound"
    if lse is not None:
        empty = np.isneginf(ref_lse)
        np.testing.assert_array_equal(np.isneginf(lse), empty)
        assert (np.abs(lse - ref_lse)[~empty] <= (eps + 1e-5 * (1 + np.abs(ref_lse)))[~empty]).all()
    if weights is not None:
        e = eps.reshape(nq, kv, -1).max(-1)[..., None]
        assert (np.abs(weights - ref_w) <= (2 * e + 2.0 ** -15) * ref_w + 1e-7).all()
    return float(np.max(err / np.maximum(bound, 1e-30)))
