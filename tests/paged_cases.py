"""Inputs and bounds shared by the tests of the paged cache and of the dense attentions."""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def normal(seed, *shape, dt, mean=0.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) + mean).to(dt).to(device)


def i32(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def cu(lens):
    return [0, *np.cumsum(lens).tolist()]


def random_parents(seed, nodes):
    rng = np.random.default_rng(seed)
    return [int(rng.integers(max(-1, i - 6), i)) if i else -1 for m in nodes for i in range(m)]


def random_pool(seed, kv, pages, dt, device="cuda"):
    return (normal(seed, kv, 64 * pages, 128, dt=dt, device=device),
            normal(seed + 1, kv, pages, 128, 64, dt=dt, mean=0.25, device=device))


def random_table(seed, n_tokens, pages, width):
    rng = np.random.default_rng(seed)
    order, at = rng.permutation(pages).tolist(), 0
    table = []
    for n in n_tokens:
        nb = (n + 63) // 64
        table.append(order[at:at + nb] + [-1] * (width - nb))
        at += nb
    assert at <= pages
    return table


def check_attention(out, lse, want, dt):
    """out and lse against (out, lse, mass, logit) in 64 bits, within the sum of the roundings:
    weights rounded to `dt` for their product with V (half a step of each: `HALF` of the mass, and in fp16 half its
    least step, 2^-25, for a weight below its normal range, times what they weigh; the largest weight is at least
    1); a logit's 128 fp32 additions and its scaling, 2^-17 of the sum of magnitudes, which a weight's numerator and
    denominator both carry; 2^-14 for fp32 sums over up to 2^14 terms of 16 keys each; half a step of
    the output's type."""
    ref, ref_lse, mass, logit = (x.cpu() for x in want)
    got, got_lse = out.double().cpu(), None if lse is None else lse.double().cpu()
    eps = 2.0 ** -17 * logit + 2.0 ** -20
    tiny = 2.0 ** -25 * 64 * mass.amax(-1, keepdim=True) if dt == torch.float16 else 0.0
    bound = (HALF[dt] + 2 * eps[..., None] + 2.0 ** -14) * mass + HALF[out.dtype] * ref.abs() + tiny + 2.0 ** -25
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    worst = float((err / bound.clamp(min=1e-30)).max()) if err.numel() else 0.0
    assert worst <= 1, f"out off by {worst:.3g} x its bound"
    if got_lse is not None:
        empty = torch.isneginf(ref_lse)
        assert torch.equal(torch.isneginf(got_lse), empty)
        assert ((got_lse - ref_lse).abs()[~empty] <= (eps + 1e-5 * (1 + ref_lse.abs()))[~empty]).all()
    return worst
