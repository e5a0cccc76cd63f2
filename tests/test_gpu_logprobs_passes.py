"""Whole-vocabulary alternatives over many short passes: the rows a block works on change every few
microseconds while its bound warps read and publish their bounds.

The inputs are multiples of 2^-3 and 2^-6, small, so logits are exact in fp32 in any order and the
alternatives, ties to the lowest token, have to be equal to those of a sort in 64 bits.
"""
import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def grid(n, H, V, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = (torch.randint(-8, 9, (n, H), device="cuda", generator=g) / 8.0).to(BF)
    W = (torch.randint(-16, 17, (V, H), device="cuda", generator=g) / 64.0).to(BF)
    return h, W


def best(h, W, top):
    val, ids = torch.sort(h.double() @ W.double().t(), dim=1, descending=True, stable=True)
    return ids[:, :top].to(torch.int32)


@pytest.mark.parametrize("n,V,top", [(8192, 300, 32), (8192, 1000, 20), (5000, 2049, 8)])
def test_alternatives_of_many_short_passes(n, V, top):
    h, W = grid(n, 64, V, seed=V)
    want = best(h, W, top)
    ws = None
    for _ in range(5):
        r = blink.blink_token_logprobs(h, W, top=top, ws=ws)
        ws = r["ws"]
        assert torch.equal(r["top_ids"], want)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK


@pytest.mark.parametrize("top", [5, 20, 32])
def test_a_bound_of_one_pass_does_not_reach_the_next(top):
    """Every logit of every second 1024 rows is 128 lower than all logits of the others: with the bound of a row
    of the pass before, such a row would lose its alternatives."""
    n, H, V = 8192, 64, 3000
    h, W = grid(n, H, V, seed=top)
    W[:, 0] = 1.0
    h[:, 0] = torch.where(torch.arange(n, device="cuda") // 1024 % 2 == 0, 64.0, -64.0).to(BF)
    want = best(h, W, top)
    for _ in range(5):
        assert torch.equal(blink.blink_token_logprobs(h, W, top=top)["top_ids"], want)
