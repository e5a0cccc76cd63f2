"""Attention weight per prefix key against the formula in 64 bits.

Tolerance, relative to each weight.  A term is exp(x), x = scale s - lse.  s is a sum of d exact bf16
products accumulated in fp32, each addition off by at most one unit in the last place (2^-23, the
accumulator may truncate) of the running sum, which sum |q_i k_i| bounds; scaling, the bias and the
exponent's argument add a few roundings of |scale s| and |lse|, and exp2 itself 2^-22.  The terms are
added in tiles of 256 columns (chains of at most 128), and at most 256 tiles and pieces in a row here.
"""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def make(rows, P, Hq, Hkv, d, seed=0, lse_pad=0, k_pad=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (spread * torch.randn(rows, Hq, d, device="cuda", generator=g)).to(BF)
    arena = torch.randn(P + 3, Hkv * d + k_pad, device="cuda", generator=g).to(BF)
    k = arena[2:2 + P, :Hkv * d].unflatten(1, (Hkv, d)) if k_pad else arena[2:2 + P].view(P, Hkv, d)
    s = torch.einsum("thgd,phd->hgtp", q.double().view(rows, Hkv, Hq // Hkv, d), k.double()) / math.sqrt(d)
    wide = torch.full((Hq, rows + lse_pad), float("nan"), device="cuda")
    lse = wide[:, lse_pad:]
    lse.copy_(torch.logsumexp(s, dim=-1).view(Hq, rows) + 0.05)
    return q, k, lse


def ref(q, k, lse, scale=None):
    rows, Hq, d = q.shape
    Hkv = k.shape[1]
    scale = 1 / math.sqrt(d) if scale is None else scale
    qd, kd = q.double().view(rows, Hkv, Hq // Hkv, d), k.double()
    s = torch.einsum("thgd,phd->hgtp", qd, kd) * scale
    x = s - lse.double().view(Hkv, Hq // Hkv, rows, 1)
    dead = torch.isneginf(lse).view(Hkv, Hq // Hkv, rows, 1)
    w = torch.where(dead, torch.zeros_like(x), x.exp()).sum((1, 2))
    mag = float(torch.nan_to_num(torch.einsum("thgd,phd->hgtp", qd.abs(), kd.abs())).max()) * scale
    big = float(torch.nan_to_num(lse, neginf=0.0).abs().max())
    tol = 2.0**-23 * ((d + 2) * mag + 4 * (mag + big) + 2 + 128 + 256)
    return w, tol


def check(got, q, k, lse, scale=None, add=None):
    want, tol = ref(q, k, lse, scale)
    if add is not None:
        want, tol = want + add.double(), tol + 2.0**-23
    assert got.dtype == torch.float32 and got.shape == want.shape
    err = ((got.double() - want).abs() / want.abs().clamp(min=1e-30)).max()
    assert float(err) <= tol, (float(err), tol)


@pytest.mark.parametrize("rows,P,Hq,Hkv,d", [
    (1, 1, 1, 1, 64), (1, 1, 4, 2, 128), (60, 64, 4, 2, 64), (1, 2048, 32, 8, 128), (5, 127, 8, 8, 64),
    (3, 129, 6, 2, 128), (4, 1300, 16, 2, 64), (8, 700, 8, 2, 128), (9, 700, 8, 2, 128), (32, 515, 3, 3, 128), (64, 256, 4, 1, 128), (65, 257, 4, 1, 128), (17, 1000, 40, 8, 128), (51, 511, 5, 1, 64),
    (2, 300, 128, 1, 64), (3, 300, 127, 1, 128), (700, 513, 7, 1, 128), (257, 3000, 2, 2, 64), (130, 5000, 28, 4, 128),
    (1000, 700, 16, 2, 64)])
def test_against_formula(rows, P, Hq, Hkv, d):
    q, k, lse = make(rows, P, Hq, Hkv, d, seed=rows + P)
    w, ws = blink.blink_prefix_key_weights(q, k, lse)
    check(w, q, k, lse)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK


def test_strided_arena_lse_slice_output_view_and_scale():
    q, k, lse = make(37, 333, 8, 2, 128, seed=4, lse_pad=11, k_pad=64)
    full = torch.full((2, 400), -7.0, device="cuda")
    w, _ = blink.blink_prefix_key_weights(q, k, lse, scale=0.05, out=full[:, 20:353])
    # lse was made for the default scale: for a smaller one the terms are smaller, the formula the same
    check(w, q, k, lse, scale=0.05)
    assert bool((full[:, :20] == -7).all()) and bool((full[:, 353:] == -7).all())


@pytest.mark.parametrize("decay", [1.0, 0.3])
def test_accumulation_in_place_and_apart(decay):
    q, k, lse = make(300, 777, 8, 2, 64, seed=9)
    prev = torch.rand(2, 777, device="cuda")
    keep = prev.clone()
    w, _ = blink.blink_prefix_key_weights(q, k, lse, prev=prev, decay=decay)
    check(w, q, k, lse, add=decay * keep.double())
    assert torch.equal(prev, keep)
    w2, _ = blink.blink_prefix_key_weights(q, k, lse, prev=prev, decay=decay, out=prev)
    assert w2.data_ptr() == prev.data_ptr() and torch.equal(w2, w)


def test_decay_zero_does_not_read_previous():
    q, k, lse = make(9, 100, 4, 2, 64)
    prev = torch.full((2, 100), float("nan"), device="cuda")
    w, _ = blink.blink_prefix_key_weights(q, k, lse, prev=prev, decay=0.0)
    check(w, q, k, lse)


@pytest.mark.parametrize("rows,Hq,Hkv,d", [(70, 4, 2, 64), (200, 10, 2, 128), (3, 8, 1, 128)])
def test_unowned_rows_add_nothing(rows, Hq, Hkv, d):
    """Rows with lse = -inf may hold anything: padding of a right-padded batch, infinities, NaN."""
    q, k, lse = make(rows, 260, Hq, Hkv, d, seed=3)
    q[0] = float("nan")
    lse[:, 0] = float("-inf")
    q[rows // 2, :, 1] = float("inf")
    lse[:, rows // 2] = float("-inf")
    w, _ = blink.blink_prefix_key_weights(q, k, lse)
    mask = torch.ones(rows, dtype=torch.bool, device="cuda")
    mask[0] = mask[rows // 2] = False
    check(w, q[mask], k, lse[:, mask])
    lse[:] = float("-inf")
    w, _ = blink.blink_prefix_key_weights(q, k, lse)
    assert bool((w == 0).all())


def test_nan_in_an_owned_row_stays_in_its_head():
    q, k, lse = make(40, 200, 4, 2, 64, seed=5)
    q[7, 3, 2] = float("nan")  # kv head 1
    w, _ = blink.blink_prefix_key_weights(q, k, lse)
    assert bool(w[1].isnan().all())
    check(w[:1], q[:, :2].contiguous(), k[:, :1].contiguous(), lse[:2])


def test_keys_past_the_prefix_are_not_read():
    """NaN in the arena rows around the prefix changes nothing."""
    q, k, lse = make(20, 130, 4, 2, 64, seed=6)
    arena = torch.full((400, 2, 64), float("nan"), dtype=BF, device="cuda")
    arena[100:230] = k
    w, _ = blink.blink_prefix_key_weights(q, arena[100:230], lse)
    check(w, q, k, lse)


def test_large_scores_and_small_weights():
    """Scores of several hundred with their lse: the largest weight is 1, the others underflow to 0."""
    q, k, lse = make(16, 300, 2, 1, 64, seed=8, spread=60.0)
    w, _ = blink.blink_prefix_key_weights(q, k, lse)
    want, tol = ref(q, k, lse)
    assert float(lse.abs().max()) > 100
    assert float((w.double() - want).abs().max()) <= 32 * tol  # 32 terms of at most 1 per key
    assert abs(float(w.sum()) - float(want.sum())) <= 32 * tol  # all terms add up to 32 e^-0.05


def test_weights_sum_to_rows_and_repeat_bitwise():
    """Each (row, head) spreads a weight of e^-0.05 over the prefix; the same call gives the same bits."""
    q, k, lse = make(333, 1500, 8, 4, 128, seed=11)
    ws = None
    first = None
    for _ in range(3):
        w, ws = blink.blink_prefix_key_weights(q, k, lse, ws=ws)
        first = w if first is None else first
        assert torch.equal(w, first)
    assert torch.allclose(first.double().sum(1), torch.full((4,), 333 * 2 * math.exp(-0.05), dtype=torch.float64,
                                                            device="cuda"), rtol=1e-4)


def test_own_stream_and_graph_replay():
    q, k, lse = make(150, 900, 8, 2, 128, seed=12)
    want, _ = blink.blink_prefix_key_weights(q, k, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w, _ = blink.blink_prefix_key_weights(q, k, lse, stream=side)
    side.synchronize()
    assert torch.equal(w, want)
    ws = blink.new_workspace(blink.key_weights_workspace_bytes(150, 900, 8, 2, 128), "cuda")
    acc = torch.zeros(2, 900, device="cuda")
    blink.blink_prefix_key_weights(q, k, lse, prev=acc, decay=1.0, out=acc, ws=ws)  # lazy loading before the capture
    acc.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blink.blink_prefix_key_weights(q, k, lse, prev=acc, decay=1.0, out=acc, ws=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.allclose(acc, 3 * want, rtol=1e-6)


def test_two_graphs_of_one_workspace_and_two_streams():
    """Replays in turn share a workspace; calls at the same time have one each."""
    cases = [make(700, 513, 8, 2, 128, seed=31), make(90, 3000, 16, 4, 64, seed=32)]
    want = [blink.blink_prefix_key_weights(*c)[0].clone() for c in cases]
    for c, w in zip(cases, want):
        check(w, *c)
    ws = blink.new_workspace(max(blink.key_weights_workspace_bytes(c[0].shape[0], c[1].shape[0], c[0].shape[1], c[1].shape[1],
                                                                   c[0].shape[2]) for c in cases), "cuda")
    outs = [torch.empty_like(w) for w in want]
    graphs = []
    for c, out in zip(cases, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            blink.blink_prefix_key_weights(*c, out=out, ws=ws)
        graphs.append(graph)
    for _ in range(3):
        for graph, out, w in zip(graphs, outs, want):
            out.fill_(-1.0)
            graph.replay()
            assert torch.equal(out, w)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, c, out in zip(streams, cases, outs):
            blink.blink_prefix_key_weights(*c, out=out, stream=s)
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out, w)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
