"""Precision of the whole-vocabulary log probabilities over long rows, against 64 bits.

A logit is added up in the tensor core over at most 512 of H (256 for up to 32 rows), 16 products a step, and these
parts are added to nearest.  A step cuts the sum it leaves off: at most 2^-22 of it (one unit in the last
place for the result and one for the products, which are aligned to it).  So the error of a logit is
bounded by 2^-22 times the sum of its own partial sums after every step, taken here in 64 bits, and by
2^-24 of the running sum for each part.  Where all products have one sign that is 3.9e-6 of the logit
whatever H is.  (One sum over all of H, tried once: lse off by 5.7e-5 at H = 2560 and 1.8e-4 at 5120, where
logits of 12 allow 3.4e-5 to 5.7e-5 in all.)

lse and entropy carry these errors weighted by the probabilities.  On top come, for sums of
2^x: 2^-22 for exp2, three roundings of x, at most 32 additions in a thread and 32 more until the row is
joined, each to nearest, and a few roundings of the results.
"""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
V = 5003


def logits_and_bound(h, W, part):
    """[n, V] logits in 64 bits, and the bound of each one's error."""
    n, H = h.shape
    hd, wd = h.double(), W.double().t().contiguous()
    z = torch.zeros(n, W.shape[0], dtype=torch.float64, device="cuda")
    steps = torch.zeros_like(z)
    joins = torch.zeros_like(z)
    for a in range(0, H, part):
        run = torch.zeros_like(z)
        for b in range(a, min(H, a + part), 16):
            run += hd[:, b:b + 16] @ wd[b:b + 16]
            steps += run.abs()
        z += run
        joins += z.abs()
    return z, 2.0**-22 * steps + 2.0**-24 * joins


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("n,H", [(1, 2560), (20, 2560), (20, 5120), (64, 2560), (100, 5120), (200, 2560), (300, 5120)])
def test_long_rows(n, H, one_sign):
    g = torch.Generator(device="cuda").manual_seed(n + H)
    if one_sign:
        h = (0.5 + torch.rand(n, H, device="cuda", generator=g)).to(BF)
        W = (12.0 / H * (0.5 + torch.rand(V, H, device="cuda", generator=g))).to(BF)
    else:
        h = torch.randn(n, H, device="cuda", generator=g).to(BF)
        W = (0.02 * torch.randn(V, H, device="cuda", generator=g)).to(BF)
    t = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    z, dz = logits_and_bound(h, W, 256 if n <= 32 else 512)
    lse = torch.logsumexp(z, 1)
    logp = z - lse[:, None]
    p = logp.exp()
    entropy = -(p * logp).sum(1)
    x = z.max(1).values[:, None] - z
    # of ln of the sum, relative to each term: its exponent, exp2, the additions, log2 and the last product
    sums = 2.0**-24 * (3 * (p * x).sum(1) + 4 + 64 + 4 + 2 * math.log(V))
    d_lse = (p * dz).sum(1) + sums
    r = blink.blink_token_logprobs(h, W, targets=t, top=10)
    at = t.long()[:, None]
    err = (r["lse"].double() - lse).abs()
    assert bool((err <= d_lse + 2.0**-23 * lse.abs()).all()), (float(err.max()), float(d_lse.max()))
    want = torch.gather(logp, 1, at).squeeze(1)
    err = (r["logprob"].double() - want).abs()
    assert bool((err <= torch.gather(dz, 1, at).squeeze(1) + d_lse + 2.0**-22 * want.abs()).all())
    # entropy = sum p (lse - z): an error dz of a logit moves it by p (entropy + log p) dz
    moved = (p * (entropy[:, None] + logp).abs() * dz).sum(1)
    err = (r["entropy"].double() - entropy).abs()
    tol = moved + sums * (2 + (p * x).sum(1))
    assert bool((err <= tol).all()), (float(err.max()), float(tol.max()))
    mine = torch.gather(logp, 1, r["top_ids"].long())
    err = (r["top_logprobs"].double() - mine).abs()
    assert bool((err <= torch.gather(dz, 1, r["top_ids"].long()) + d_lse[:, None] + 2.0**-22 * mine.abs()).all())


@pytest.mark.parametrize("n,H", [(20, 1344), (100, 1344), (129, 1032), (300, 1344), (300, 5064), (200, 2888)])
def test_several_parts_of_exact_logits(n, H):
    """Logits that are exact in any order, over several parts of H, the last of an odd number of 64-wide blocks."""
    g = torch.Generator(device="cuda").manual_seed(H)
    h = (torch.randint(-8, 9, (n, H), device="cuda", generator=g) / 8.0).to(BF)
    W = (torch.randint(-16, 17, (V, H), device="cuda", generator=g) / 64.0).to(BF)
    val, ids = torch.sort(h.double() @ W.double().t(), dim=1, descending=True, stable=True)
    r = blink.blink_token_logprobs(h, W, top=32)
    assert torch.equal(r["top_ids"], ids[:, :32].to(torch.int32))
    gap = r["top_logprobs"].double()[:, :1] - r["top_logprobs"].double()
    want = val[:, :1] - val[:, :32]  # differences of exact logits: the roundings of the two log probabilities
    assert float(((gap - want).abs() - 2.0**-22 * (want + r["top_logprobs"].double()[:, :1].abs())).max()) <= 0
