"""The paged operators together, as a program uses them: a prefix rotated into 8-bit pages once, questions that attend
to it and are read out, then tokens one by one, eagerly and in a captured graph."""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402


def test_prefix_into_pages_then_questions_and_readout():
    g = ph.gen(31)
    Hq, Hkv, d, page, P, H, V = 8, 2, 64, 32, 333, 512, 400
    tails = [5, 1, 17, 40]
    rows = sum(tails)
    cu_l = [sum(tails[:i]) for i in range(len(tails) + 1)]
    cu = torch.tensor(cu_l, dtype=torch.int32, device="cuda")
    turns, amp = blink.blink_rope_table(d, 10000.0, scaling="by_turns", factor=2.0, original=256)
    theta, _ = ph.frequencies(d, 10000.0, "by_turns", 2.0, 256, 1.0, 4.0)
    k_pre, v_pre = (ph.randn(g, P, Hkv, d).to(torch.bfloat16) for _ in range(2))
    q, k, v = (ph.randn(g, rows, n, d).to(torch.bfloat16) for n in (Hq, Hkv, Hkv))
    table, total = ph.table_for(g, [P], page)
    cache = blink.blink_paged_cache(total, page, Hkv, d)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # the prefix arrives in two pieces that meet inside a page
    for a, b in ((0, 200), (200, P)):
        blink.blink_paged_append(k_pre[a:b], v_pre[a:b], cache, table, i32(0, b - a), i32(a), b - a, turns=turns, amplitude=amp)
    pos = torch.cat([torch.arange(P, P + t) for t in tails]).to(torch.int32).cuda()
    qr, kr = blink.blink_rope(q, k, pos, turns, amplitude=amp)
    out, lse, ws = blink.blink_paged_prefix_tail_attention(qr, cache, table, [P], kr, v, cu, len(tails), max(tails), want_lse=True)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    # 64 bits from the unrotated inputs: 8-bit keys and values are off by half a step, 2^-4 of a value, which the
    # softmax over 333 keys averages; the whole output stays within 2^-4 of its size
    kd, _ = ph.rotate(k_pre, torch.arange(P, device="cuda"), theta, 1.0, False)
    qd, _ = ph.rotate(q, pos, theta, 1.0, False)
    td, _ = ph.rotate(k, pos, theta, 1.0, False)
    want = torch.empty(rows, Hq, d, dtype=torch.float64, device="cuda")
    for b in range(len(tails)):
        for i in range(cu_l[b], cu_l[b + 1]):
            kk = torch.cat([kd, td[cu_l[b]:i + 1]]).transpose(0, 1)
            vv = torch.cat([v_pre, v[cu_l[b]:i + 1]]).double().transpose(0, 1)
            want[i] = ph.attend(qd[i], kk, vv, 1 / math.sqrt(d))[0]
    assert float((out.double() - want).norm() / want.norm()) <= 2.0 ** -4
    hidden = out.reshape(rows, H)
    unembed = (0.02 * ph.randn(g, V, H)).to(torch.bfloat16)
    off, ids = i32(0, 3, 5, 9, 12), torch.arange(12, dtype=torch.int32, device="cuda")
    probs, _ = blink.blink_label_readout(hidden, cu[1:] - 1, unembed, off, ids, 1.0)
    z = hidden[(cu[1:] - 1).long()].double() @ unembed[:12].double().t()
    for b in range(4):
        a, e = int(off[b]), int(off[b + 1])
        assert float((probs[a:e].double() - torch.softmax(z[b, a:e], 0)).abs().max()) <= 1e-3


def test_tokens_one_by_one_eagerly_and_in_a_graph():
    """Each step rotates, appends and attends; the captured step follows the growing lengths and gives the same bits."""
    g = ph.gen(32)
    S, Hq, Hkv, d, page, steps = 3, 8, 2, 64, 16, 37
    starts = [0, 15, 250]
    room = [a + steps for a in starts]
    table, total = ph.table_for(g, room, page)
    turns, amp = blink.blink_rope_table(d)

    def fresh():
        c = ph.new_cache(g, total, Hkv, page, d)
        ph.fill(ph.gen(77), c, table, starts)
        return c

    x = [tuple(ph.randn(g, S, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv)) for _ in range(steps)]
    one = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    ws_a = blink.new_workspace(blink.paged_append_workspace_bytes(), "cuda")
    ws_t = blink.new_workspace(blink.paged_token_attention_workspace_bytes(S, 1, max(room), Hq, Hkv, d), "cuda")

    def step(cache, q, k, v, length):
        qr, _ = blink.blink_rope(q, None, length, turns, amplitude=amp)
        blink.blink_paged_append(k, v, cache, table, one, length, 1, turns=turns, amplitude=amp, ws=ws_a)
        length += 1
        out, lse, _ = blink.blink_paged_token_attention(qr.view(S, 1, Hq, d), cache, table, length, max(room), want_lse=True, ws=ws_t)
        return out, lse

    eager, cache, length = [], fresh(), torch.tensor(starts, dtype=torch.int32, device="cuda")
    for t in range(steps):
        out, lse = step(cache, *x[t], length)
        if t in (0, 1, steps - 1):
            lens = [a + t + 1 for a in starts]
            qr, _ = blink.blink_rope(x[t][0], None, length - 1, turns, amplitude=amp)
            ph.check_attention(out, lse, ph.token_reference(qr.view(S, 1, Hq, d), cache, table, lens))
        eager.append((out.clone(), lse.clone()))
    assert blink.blink_read_device_status(ws_a) == blink.blink_read_device_status(ws_t) == blink.BLINK_OK

    cache2, length2 = fresh(), torch.tensor(starts, dtype=torch.int32, device="cuda")
    q, k, v = (torch.empty_like(y) for y in x[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(cache2, q, k, v, length2)
    for t in range(steps):
        q.copy_(x[t][0]), k.copy_(x[t][1]), v.copy_(x[t][2])
        graph.replay()
        assert torch.equal(out, eager[t][0]) and torch.equal(lse, eager[t][1])
    assert all(torch.equal(cache[n].view(torch.uint8), cache2[n].view(torch.uint8)) for n in cache)


def test_single_token_equals_a_one_token_tail():
    """A token appended and then attended to against the same token as a question's tail: keys and values differ by
    their rounding to 8 bits in that one place."""
    g = ph.gen(33)
    Hq, Hkv, d, page, P = 8, 2, 128, 64, 700
    table, total = ph.table_for(g, [P + 1], page)
    cache = blink.blink_paged_cache(total, page, Hkv, d)
    ph.fill(g, cache, table, [P])
    q, k, v = (ph.randn(g, 1, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tail, lse_t, _ = blink.blink_paged_prefix_tail_attention(q, cache, table, [P], k, v, i32(0, 1), 1, 1, want_lse=True)
    blink.blink_paged_append(k, v, cache, table, i32(0, 1), i32(P), 1)
    tok, lse, _ = blink.blink_paged_token_attention(q.view(1, 1, Hq, d), cache, table, i32(P + 1), P + 1, want_lse=True)
    kk, vv = (torch.cat([ph.values(cache, n, table[0], P), x.double().transpose(0, 1)], dim=1) for n, x in (("k", k), ("v", v)))
    z = torch.einsum("hd,hnd->hn", q[0].double(), kk.repeat_interleave(4, 0)) / math.sqrt(d)
    w = torch.softmax(z, dim=1)[:, -1]  # the weight of the token itself
    moved = 2.0 ** -4 * torch.einsum("hd,hd->h", q[0].double().abs(), k[0].double().abs().repeat_interleave(4, 0)) / math.sqrt(d)
    grow = w * torch.expm1(moved)  # how far the weights can go
    size = torch.cat([vv.abs()], dim=1).amax(dim=(1, 2)).repeat_interleave(4)
    assert bool(((lse[:, 0].double() - lse_t[:, 0].double()).abs() <= grow + 1e-3).all())
    err = (tok[0, 0].double() - tail[0].double()).abs().amax(dim=1)
    assert bool((err <= (2 * grow + 2.0 ** -4 * w) * size + 2e-2 * tail[0].double().abs().amax(dim=1)).all())
