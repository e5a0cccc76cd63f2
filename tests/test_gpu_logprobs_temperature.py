"""Whole-vocabulary log probabilities at small and large temperatures, where logits divided by the temperature
have no digits left behind the point, against 64 bits.

Logits are multiples of 2^-9 below 2^15, exact in fp32, as are their differences, and the temperatures
are powers of two.  So the scaled difference of two logits is off by the rounding of log2(e) and of one product,
and in nats by those of ln 2 and one more: 4 x 2^-24 of it.  The sum of the probabilities: exponents
off by 2 x 2^-24 of their size, whose average over a distribution of V tokens is below log2 V; exp2 2^-22;
chains of at most 1024 additions of 2^-24; log2 and its scaling a few more of at most log2 V.
"""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
V, TOP = 3001, 20
SUM = 2.0**-24 * (1024 + 4 + 12 * math.log2(V))  # of ln of the sum of the probabilities
EACH = 4 * 2.0**-24


@pytest.mark.parametrize("n", [3, 100, 300])
@pytest.mark.parametrize("log2_t", [20, 0, -4, -10, -16, -20, -24, -32, -64, -100, -116, -119])
def test_powers_of_two(n, log2_t):
    T = 2.0**log2_t
    g = torch.Generator(device="cuda").manual_seed(n)
    h = (torch.randint(-8, 9, (n, 64), device="cuda", generator=g) / 8.0).to(BF)
    W = (torch.randint(-16, 17, (V, 64), device="cuda", generator=g) / 64.0).to(BF)
    t = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    z = h.double() @ W.double().t() / T
    t[0] = int(z[0].argmax())  # the best token of a row
    zmax = z.max(1).values
    sums = (z - zmax[:, None]).exp().sum(1).log()  # apart from zmax: of 10^20 not even 64 bits hold a ln 2
    lse = zmax + sums
    logp = z - zmax[:, None] - sums[:, None]
    p = logp.exp()
    entropy = -(p * logp).sum(1)
    _, ids = torch.sort(z, dim=1, descending=True, stable=True)
    assert float(z.abs().max()) < 1e38
    r = blink.blink_token_logprobs(h, W, targets=t, temperature=T, top=TOP)
    assert torch.equal(r["top_ids"], ids[:, :TOP].to(torch.int32))
    want = torch.gather(logp, 1, ids[:, :TOP])
    assert bool(((r["top_logprobs"].double() - want).abs() <= EACH * want.abs() + SUM).all())
    want = torch.gather(logp, 1, t.long()[:, None]).squeeze(1)
    assert bool(((r["logprob"].double() - want).abs() <= EACH * want.abs() + SUM).all())
    assert bool(((r["lse"].double() - lse).abs() <= EACH * lse.abs() + SUM).all())
    # entropy = ln s - u / s in nats, both sums with the error of SUM, the second times what it is: at most ln V
    assert bool(((r["entropy"].double() - entropy).abs() <= SUM * (2 + 2 * math.log(V))).all())
    assert bool((r["logprob"] <= SUM).all()) and bool((r["entropy"] >= -SUM).all())


def test_large_logits():
    """Logits of 10^9 and more at temperature 1: the best tokens and their differences are still exact."""
    h = torch.zeros(200, 64, dtype=BF, device="cuda")
    h[:, 0] = 2.0**20
    W = torch.zeros(V, 64, dtype=BF, device="cuda")
    W[:, 0] = (torch.arange(V, device="cuda") % 64 * 16).to(BF)
    W[77, 0] = W[1001, 0] = 2048.0
    t = torch.full((200,), 77, dtype=torch.int32, device="cuda")
    r = blink.blink_token_logprobs(h, W, targets=t, top=2)
    assert r["top_ids"].tolist() == [[77, 1001]] * 200
    for key in ("logprob", "top_logprobs"):
        assert float((r[key] + math.log(2)).abs().max()) <= SUM
    assert float((r["entropy"] - math.log(2)).abs().max()) <= SUM * 4
    assert float((r["lse"].double() / (2.0**31 + math.log(2)) - 1).abs().max()) <= EACH
