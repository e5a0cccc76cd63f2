"""Whole-vocabulary log probabilities against the formulas in 64 bits.

Two kinds of inputs.  On the grid (hidden states and rows multiples of 2^-3 and 2^-6, small) every product
and partial sum is a multiple of 2^-9 below 2^15, so fp32 logits are exact in any order and the
alternatives, ties included, have to be equal.  Normal inputs: a logit is a sum of H exact products in
fp32, each addition off by at most 2^-23 of the running sum, which sum |h w| bounds; lse and the
probabilities it enters carry the largest such error once more; the scaled logits, exp2, log2 and the
sum over the vocabulary (chains of at most 1024) add a few roundings of |z| + |lse|.
"""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def normal(n, H, V, seed=0, std=0.05, rows=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(rows or n, H, device="cuda", generator=g).to(BF)
    W = (std * torch.randn(V, H, device="cuda", generator=g)).to(BF)
    t = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    return h, W, t


def grid(n, H, V, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = (torch.randint(-8, 9, (n, H), device="cuda", generator=g) / 8.0).to(BF)
    W = (torch.randint(-16, 17, (V, H), device="cuda", generator=g) / 64.0).to(BF)
    W[torch.rand(V, H, device="cuda", generator=g) < 0.7] = 0  # few distinct logits: many ties
    t = torch.randint(0, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    return h, W, t


def ref(h, W, t, T, top):
    z = h.double() @ W.double().t() / T
    lse = torch.logsumexp(z, 1)
    p = (z - lse[:, None]).exp()
    val, ids = torch.sort(z, dim=1, descending=True, stable=True)
    out = {"lse": lse, "entropy": (p * (lse[:, None] - z)).sum(1), "top_ids": ids[:, :top].to(torch.int32),
           "top_logprobs": val[:, :top] - lse[:, None]}
    if t is not None:
        out["logprob"] = torch.gather(z, 1, t.long()[:, None]).squeeze(1) - lse
    mag = float((h.abs().double() @ W.abs().double().t()).max()) / T
    zmax = float(z.abs().max())
    return out, mag, zmax


def check(r, want, mag, zmax, H, V, exact_ids, rows=slice(None)):
    eps = 2.0**-23
    dz = eps * (H * mag + 4 * zmax)                      # one logit
    dl = 2 * dz + eps * (1024 + 16 + 4 * (zmax + math.log(V)))  # a log probability: its logit and the lse
    dH = dl * (2 + 2 * zmax + math.log(V))               # entropy: probabilities off by dl, weights up to the spread
    for key, tol in (("lse", dl), ("logprob", dl), ("entropy", dH), ("top_logprobs", dl)):
        if key in want and r[key] is not None:
            err = float((r[key][rows].double() - want[key]).abs().max())
            assert err <= tol, (key, err, tol)
    if r["top_ids"] is not None and exact_ids:
        assert torch.equal(r["top_ids"][rows], want["top_ids"])


@pytest.mark.parametrize("n,H,V,top,T", [
    (1, 8, 1, 1, 1.0), (1, 8, 7, 5, 1.0), (4, 256, 1024, 5, 1.0), (1, 64, 255, 20, 0.7), (2, 72, 256, 32, 1.3),
    (3, 200, 257, 0, 1.0), (127, 64, 1000, 8, 1.0), (128, 128, 513, 9, 1.0), (129, 136, 4000, 3, 2.0),
    (255, 64, 3000, 1, 1.0), (256, 64, 777, 32, 1.0), (257, 264, 5001, 20, 0.5), (700, 64, 2049, 4, 1.0),
    (1300, 128, 1025, 8, 1.0), (33, 1024, 20000, 20, 1.0)])
def test_grid_inputs_exact_alternatives(n, H, V, top, T):
    h, W, t = grid(n, H, V, seed=n + H + V)
    r = blink.blink_token_logprobs(h, W, targets=t, temperature=T, top=top)
    want, mag, zmax = ref(h, W, t, T, top)
    check(r, want, 0.0, zmax, H, V, True)
    assert blink.blink_read_device_status(r["ws"]) == blink.BLINK_OK


@pytest.mark.parametrize("n,H,V,T", [(1, 2560, 30011, 1.0), (64, 2560, 20000, 0.7), (300, 1000, 9999, 1.0),
                                     (40, 5120, 4097, 1.0)])
def test_normal_inputs(n, H, V, T):
    h, W, t = normal(n, H, V, seed=n, std=0.02)
    r = blink.blink_token_logprobs(h, W, targets=t, temperature=T, top=10)
    want, mag, zmax = ref(h, W, t, T, 10)
    check(r, want, mag, zmax, H, V, False)
    # the alternatives: each one's own logit, in order, none better left out (up to the logits' error)
    dz = 2.0**-22 * (H * mag + 4 * zmax)
    z = h.double() @ W.double().t() / T
    mine = torch.gather(z, 1, r["top_ids"].long())
    assert float((mine - want["top_logprobs"] - want["lse"][:, None]).abs().max()) <= dz


def test_row_idx_gathers_strided_rows():
    big = torch.randn(50, 512, device="cuda").to(BF)
    h = big[:, :264]
    _, W, _ = normal(1, 264, 900, seed=2)
    idx = torch.tensor([49, 0, 7, 7, 31], dtype=torch.int32, device="cuda")
    t = torch.tensor([0, 899, 5, 5, 450], dtype=torch.int32, device="cuda")
    r = blink.blink_token_logprobs(h, W, targets=t, row_idx=idx, top=4)
    want, mag, zmax = ref(h[idx.long()], W, t, 1.0, 4)
    check(r, want, mag, zmax, 264, 900, False)
    assert torch.equal(r["top_ids"][2], r["top_ids"][3]) and float(r["logprob"][2]) == float(r["logprob"][3])
    direct = blink.blink_token_logprobs(h, W, top=4)  # all rows, strided, no targets
    assert direct["logprob"] is None
    assert torch.equal(direct["top_ids"][idx.long()], r["top_ids"])


def test_peaked_and_flat_distributions():
    """All logits equal: entropy ln V and the lowest ids; one logit far above the rest: entropy 0."""
    h = torch.zeros(2, 64, dtype=BF, device="cuda")
    h[1, 0] = 16.0
    W = torch.zeros(1500, 64, dtype=BF, device="cuda")
    W[1234, 0] = 16.0
    t = torch.tensor([3, 1234], dtype=torch.int32, device="cuda")
    r = blink.blink_token_logprobs(h, W, targets=t, top=6)
    assert r["top_ids"][0].tolist() == [0, 1, 2, 3, 4, 5]
    assert r["top_ids"][1].tolist() == [1234, 0, 1, 2, 3, 4]
    assert abs(float(r["entropy"][0]) - math.log(1500)) < 1e-5 and abs(float(r["entropy"][1])) < 1e-5
    assert float(r["logprob"][1]) == 0.0 and abs(float(r["logprob"][0]) + math.log(1500)) < 1e-5
    assert abs(float(r["top_logprobs"][1][1]) + 256.0) < 1e-4


def test_no_target_bad_target_and_bad_row():
    h, W, _ = normal(6, 64, 300, seed=3)
    idx = torch.tensor([0, 1, 2, 6, -1, 5], dtype=torch.int32, device="cuda")
    t = torch.tensor([-1, 300, 7, 8, 9, -2], dtype=torch.int32, device="cuda")
    r = blink.blink_token_logprobs(h, W, targets=t, row_idx=idx, top=3)
    lp = r["logprob"].tolist()
    assert [math.isnan(x) for x in lp] == [True, True, False, True, True, True]
    good = torch.tensor([0, 1, 2, 5], device="cuda")
    want, mag, zmax = ref(h[good], W, None, 1.0, 3)
    check(r, want, mag, zmax, 64, 300, False, rows=good)
    for row in (3, 4):
        assert r["top_ids"][row].tolist() == [-1, -1, -1] and math.isnan(float(r["entropy"][row]))
        assert math.isnan(float(r["lse"][row])) and bool(r["top_logprobs"][row].isnan().all())
    assert blink.blink_read_device_status(r["ws"]) == blink.BLINK_DEVICE_FLAG
    r = blink.blink_token_logprobs(h, W, targets=torch.full((6,), -1, dtype=torch.int32, device="cuda"), ws=r["ws"])
    assert bool(r["logprob"].isnan().all()) and bool(r["lse"].isfinite().all())
    assert blink.blink_read_device_status(r["ws"]) == blink.BLINK_OK  # -1 is no error


def test_nan_rows_stay_apart():
    h, W, t = normal(200, 64, 600, seed=4)
    h[130, 5] = float("nan")
    r = blink.blink_token_logprobs(h, W, targets=t, top=2)
    keep = torch.arange(200, device="cuda") != 130
    want, mag, zmax = ref(h[keep], W, t[keep], 1.0, 2)
    check(r, want, mag, zmax, 64, 600, False, rows=keep)
    assert math.isnan(float(r["lse"][130])) and math.isnan(float(r["entropy"][130]))
    assert r["top_ids"][130].tolist() == [-1, -1]


def test_ascending_and_descending_logits():
    """The order in which the best tokens are met does not matter."""
    V, H = 5000, 64
    W = torch.zeros(V, H, dtype=BF, device="cuda")
    i = torch.arange(V, device="cuda")
    W[:, 0], W[:, 1] = (i // 128).to(BF), (i % 128).to(BF)  # exact in bf16
    h = torch.zeros(2, H, dtype=BF, device="cuda")
    h[0, 0], h[0, 1] = 2.0, 1 / 64.0   # z = i / 64: ascending
    h[1, 0], h[1, 1] = -2.0, -1 / 64.0
    r = blink.blink_token_logprobs(h, W, top=32)
    assert r["top_ids"][0].tolist() == list(range(V - 1, V - 33, -1))
    assert r["top_ids"][1].tolist() == list(range(32))


def test_agrees_with_the_label_readout():
    """The labels' logits of blink_label_readout minus lse are their whole-vocabulary log probabilities."""
    h, W, _ = normal(3, 256, 1024, seed=6)
    off = torch.tensor([0, 2, 5, 9], dtype=torch.int32, device="cuda")
    ids = torch.tensor([3, 9, 1, 2, 3, 100, 200, 300, 1023], dtype=torch.int32, device="cuda")
    idx = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    z = torch.empty(9, device="cuda")
    blink.blink_label_readout(h, idx, W, off, ids, 1.0, logits=z)
    row = torch.tensor([2, 2, 0, 0, 0, 1, 1, 1, 1], dtype=torch.int32, device="cuda")
    r = blink.blink_token_logprobs(h, W, targets=ids, row_idx=row)
    assert float((z - r["lse"] - r["logprob"]).abs().max()) < 1e-4


def test_repeat_bitwise_own_stream_and_graph():
    h, W, t = normal(300, 512, 7001, seed=7)
    idx = torch.randperm(300, device="cuda").to(torch.int32)
    r = blink.blink_token_logprobs(h, W, targets=t, row_idx=idx, top=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r2 = blink.blink_token_logprobs(h, W, targets=t, row_idx=idx, top=5, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r3 = blink.blink_token_logprobs(h, W, targets=t, row_idx=idx, top=5)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in ("logprob", "entropy", "lse", "top_ids", "top_logprobs"):
        assert torch.equal(r[k], r2[k]) and torch.equal(r[k], r3[k]), k


@pytest.mark.parametrize("n,V,top", [(1, 5000, 20), (3, 20001, 32), (130, 3000, 9), (600, 1500, 4)])
def test_more_equal_best_logits_than_any_list_holds(n, V, top):
    """Every logit equal, or thousands of equal best ones: the lowest ids, whatever the parts are."""
    h = torch.ones(n, 64, dtype=BF, device="cuda")
    W = torch.zeros(V, 64, dtype=BF, device="cuda")
    r = blink.blink_token_logprobs(h, W, top=top)
    assert torch.equal(r["top_ids"], torch.arange(top, dtype=torch.int32, device="cuda").expand(n, top))
    W[V // 3:, 0] = 1.0
    W[5, 0] = 2.0
    r = blink.blink_token_logprobs(h, W, top=top)
    want = torch.cat([torch.tensor([5]), V // 3 + torch.arange(top - 1)]).to(torch.int32).cuda()
    assert torch.equal(r["top_ids"], want.expand(n, top))


def test_more_rows_than_one_launch():
    """8192 rows go in one launch: rows before and after the seam, gathered and direct."""
    n, H, V = 8192 + 300, 64, 700
    h, W, t = grid(n, H, V, seed=21)
    want, _, zmax = ref(h, W, t, 1.0, 3)
    r = blink.blink_token_logprobs(h, W, targets=t, top=3)
    check(r, want, 0.0, zmax, H, V, True)
    idx = torch.randperm(n, device="cuda").to(torch.int32)
    r = blink.blink_token_logprobs(h, W, targets=t[idx.long()], row_idx=idx, top=3, ws=r["ws"])
    check(r, {k: v[idx.long()] for k, v in want.items()}, 0.0, zmax, H, V, True)


def test_two_calls_at_once():
    """Two streams, a workspace each: the same results as one after the other."""
    a, b = normal(300, 512, 9000, seed=31), normal(40, 1024, 9000, seed=32)
    want = [blink.blink_token_logprobs(h, W, targets=t, top=5) for h, W, t in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [blink.blink_token_logprobs(h, W, targets=t, top=5, stream=s) for (h, W, t), s in zip((a, b), streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for k in ("logprob", "entropy", "lse", "top_ids", "top_logprobs"):
                assert torch.equal(g[k], w[k]), k


def test_fewer_numbers_than_alternatives():
    """NaN rows of the unembedding: the other tokens are listed, then -1; the sums are NaN."""
    h = torch.ones(2, 64, dtype=BF, device="cuda")
    W = torch.full((700, 64), float("nan"), dtype=BF, device="cuda")
    W[[650, 3, 300]] = torch.tensor([[0.5], [0.25], [0.5]], device="cuda").to(BF).expand(3, 64)
    r = blink.blink_token_logprobs(h, W, top=6)
    assert r["top_ids"].tolist() == [[300, 650, 3, -1, -1, -1]] * 2
    assert bool(r["lse"].isnan().all()) and bool(r["entropy"].isnan().all())
