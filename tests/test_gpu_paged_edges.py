"""The paged calls where they could go wrong between calls: pages past 4 GB, two streams at once, captured calls whose
inputs change, tables wider than the sequences, workspaces used again, one page, other devices' checks."""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_pages_past_four_gigabytes():
    """70,000 pages of 64 KB: the pages in use are the last ones, beyond 2^32 bytes of K and of V."""
    g = ph.gen(41)
    Hq, Hkv, d, page, total = 16, 8, 128, 64, 70000
    k = torch.empty(total, Hkv, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.empty_like(k)
    scale = [torch.full((total, Hkv), 120, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu) for _ in range(2)]
    cache = {"k": k, "v": v, "k_scale": scale[0], "v_scale": scale[1]}
    n = 200
    table = _i32(69999, 66001, 69990, 65537).view(1, 4)
    kk, vv = (ph.randn(g, n, Hkv, d).to(torch.bfloat16) for _ in range(2))
    turns, _ = blink.blink_rope_table(d)
    blink.blink_paged_append(kk, vv, cache, table, _i32(0, n), _i32(0), n, turns=turns)
    small = ph.new_cache(g, 4, Hkv, page, d)
    blink.blink_paged_append(kk, vv, small, _i32(0, 1, 2, 3).view(1, 4), _i32(0, n), _i32(0), n, turns=turns)
    for x in cache:
        assert torch.equal(cache[x][table[0, :3].long()].view(torch.uint8), small[x][:3].view(torch.uint8))
        assert torch.equal(cache[x][65537].view(torch.uint8)[:, :8], small[x][3].view(torch.uint8)[:, :8]) if x in "kv" else True
    q = ph.randn(g, 1, 1, Hq, d).to(torch.bfloat16)
    out, lse, _ = blink.blink_paged_token_attention(q, cache, table, _i32(n), n, want_lse=True)
    ph.check_attention(out, lse, ph.token_reference(q, cache, table, [n]))
    rows = 50
    qt, kt, vt = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    far, _, _ = blink.blink_paged_prefix_tail_attention(qt, cache, table, [n], kt, vt, _i32(0, rows), 1, rows)
    near, _, _ = blink.blink_paged_prefix_tail_attention(qt, small, _i32(0, 1, 2, 3).view(1, 4), [n], kt, vt, _i32(0, rows), 1, rows)
    assert torch.equal(far, near)


def test_two_streams_at_once():
    """Calls on two streams with a workspace each, over the same cache."""
    g = ph.gen(42)
    lens, Hq, Hkv, d, page = [9000, 300], 8, 2, 128, 64
    table, total = ph.table_for(g, lens, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, lens)
    length = _i32(*lens)
    qs = [ph.randn(g, 2, 1, Hq, d).to(torch.bfloat16) for _ in range(2)]
    want = [blink.blink_paged_token_attention(q, cache, table, length, 9000, want_lse=True)[:2] for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    need = blink.paged_token_attention_workspace_bytes(2, 1, 9000, Hq, Hkv, d)
    ws = [blink.new_workspace(need, "cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(blink.blink_paged_token_attention(qs[i], cache, table, length, 9000, want_lse=True, ws=ws[i], stream=streams[i])[:2])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) for o, l in got[i])


@pytest.mark.parametrize("rows", [3, 90])
def test_prefix_tail_captured_twice_over_one_workspace(rows):
    """Two graphs that share a workspace, replayed in turn, follow their inputs."""
    g = ph.gen(43)
    Hq, Hkv, d, page, P = 8, 2, 64, 32, 500
    table, total = ph.table_for(g, [P], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, [P])
    cu = _i32(0, 1, rows)
    ins = [tuple(ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv)) for _ in range(2)]
    ws = blink.new_workspace(blink.paged_prefix_tail_workspace_bytes([0, rows], [P], 2, Hq, Hkv, d), "cuda")
    outs, graphs = [torch.empty_like(ins[0][0]) for _ in range(2)], []

    def call(i, **kw):
        return blink.blink_paged_prefix_tail_attention(ins[i][0], cache, table, [P], ins[i][1], ins[i][2], cu, 2, rows, **kw)[0]
    for i in range(2):
        call(i, ws=ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i, ws=ws, out=outs[i])
    for step in range(4):
        for i in range(2):
            ins[i][0].copy_(ph.randn(g, rows, Hq, d))
            graphs[i].replay()
        for i in range(2):
            assert torch.equal(outs[i], call(i))


def test_wider_tables_and_bounds_than_needed():
    """A table wider than any sequence (strided rows of a larger one) and a larger max_len give the same, and a workspace
    for more serves less."""
    g = ph.gen(44)
    lens, Hq, Hkv, d, page = [100, 37, 64], 4, 2, 64, 16
    table, total = ph.table_for(g, lens, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, lens)
    q = ph.randn(g, 3, 2, Hq, d).to(torch.bfloat16)
    want = ph.token_reference(q, cache, table, lens)
    big = torch.full((3, 500), -1, dtype=torch.int32, device="cuda")
    big[:, 100:100 + table.shape[1]] = table
    wide = big[:, 100:400]
    ws = blink.new_workspace(blink.paged_token_attention_workspace_bytes(3, 2, 131072, Hq, Hkv, d), "cuda")
    for t, bound in ((table, 100), (wide, 100), (wide, 4800), (table, 131072)):
        out, lse, _ = blink.blink_paged_token_attention(q, cache, t, _i32(*lens), bound, want_lse=True, ws=ws)
        assert blink.blink_read_device_status(ws) == blink.BLINK_OK
        ph.check_attention(out, lse, want)


def test_one_page_and_one_token():
    g = ph.gen(45)
    cache = blink.blink_paged_cache(1, 128, 1, 128)
    table = _i32(0).view(1, 1)
    k, v = (ph.randn(g, 1, 1, 128).to(torch.bfloat16) for _ in range(2))
    blink.blink_paged_append(k, v, cache, table, _i32(0, 1), _i32(0), 1)
    q = ph.randn(g, 1, 1, 7, 128).to(torch.bfloat16)
    out, lse, _ = blink.blink_paged_token_attention(q, cache, table, _i32(1), 1, want_lse=True)
    kd, vd = (ph.values(cache, n, table[0], 1)[0, 0] for n in ("k", "v"))
    assert torch.equal(out[0, 0], vd.to(torch.bfloat16).expand(7, -1))
    want = (q[0, 0].double() @ kd) / math.sqrt(128)
    assert float((lse[:, 0].double() - want).abs().max()) <= 64 * ph.F32 * float((q[0, 0].double().abs() @ kd.abs()).max()) / math.sqrt(128) + 2.0 ** -20
    # nothing to do: no tokens, no keys
    none = torch.empty(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    before = cache["k"].view(torch.uint8).clone()
    blink.blink_paged_append(none, none, cache, table, _i32(0, 0), _i32(1), 0)
    assert torch.equal(cache["k"].view(torch.uint8), before)
    out, lse, ws = blink.blink_paged_token_attention(q, cache, table, _i32(0), 0, want_lse=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and blink.blink_read_device_status(ws) == blink.BLINK_OK


def test_append_repeated_is_the_same_bits_and_order_of_sequences_does_not_matter():
    g = ph.gen(46)
    n, Hkv, d, page = [70, 1, 33], 2, 64, 32
    table, total = ph.table_for(g, n, page)
    x = [ph.randn(g, sum(n), Hkv, d).to(torch.bfloat16) for _ in range(2)]
    turns, _ = blink.blink_rope_table(d)
    a, b = ph.new_cache(g, total, Hkv, page, d), ph.new_cache(g, total, Hkv, page, d)
    cu = [0, 70, 71, 104]
    blink.blink_paged_append(*x, a, table, _i32(*cu), _i32(0, 0, 0), 70, turns=turns)
    order = [2, 0, 1]
    rows = torch.cat([torch.arange(cu[s], cu[s + 1]) for s in order]).cuda()
    blink.blink_paged_append(x[0][rows], x[1][rows], b, table[order].contiguous(), _i32(0, 33, 103, 104), _i32(0, 0, 0), 70, turns=turns)
    assert all(torch.equal(a[t].view(torch.uint8), b[t].view(torch.uint8)) for t in a)


def test_codes_are_those_of_the_exact_rotation():
    """A few hundred thousand keys with values of very different sizes: every code is the nearest to the rotation in 64 bits
    (off by one only where 64 bits cannot tell: within 2^-34 of the sizes of the border)."""
    g = ph.gen(47)
    n, Hkv, d, page = 3000, 4, 128, 64
    table, total = ph.table_for(g, [n], page)
    k = (ph.randn(g, n, Hkv, d) * torch.exp(2.0 * ph.randn(g, 1, Hkv, d))).to(torch.bfloat16)
    for interleaved, rot in ((False, 128), (True, 128), (False, 122)):
        cache = ph.new_cache(g, total, Hkv, page, d)
        turns, _ = blink.blink_rope_table(rot, 500000.0)
        blink.blink_paged_append(k, k, cache, table, _i32(0, n), _i32(0), n, turns=turns, interleaved=interleaved,
                                 positions=torch.arange(n, device="cuda", dtype=torch.int32) * 41)
        # the table's own frequencies, so that only the rotation is compared
        theta = (turns.double() * (2 * math.pi / 2.0 ** 64)).tolist()
        y, size = ph.rotate(k, torch.arange(n, device="cuda") * 41, theta, 1.0, interleaved)
        at = table[0, torch.arange(n, device="cuda") // page].long()
        slot = torch.arange(n, device="cuda") % page
        scale = torch.exp2(cache["k_scale"].view(torch.uint8)[at].double() - 127)[..., None]
        got = cache["k"].view(torch.uint8)[at, :, slot].view(torch.float8_e4m3fn).double()
        lo, hi = ph.e4m3((y - size * 2.0 ** -34) / scale), ph.e4m3((y + size * 2.0 ** -34) / scale)
        assert bool(((got == lo) | (got == hi)).all())
        # the window hides little: 2^-33 of a pair's sizes against steps of 2^-4 of a value.  (The first token and the values
        # past rot are not turned: one in 16 of their 8-bit values lies on a border, and goes to the even code.)
        assert float((lo != hi)[1:, :, :rot].double().mean()) < 1e-6
        assert torch.equal(got[0], ph.e4m3(y[0] / scale[0])) and torch.equal(got[..., rot:], ph.e4m3(y / scale)[..., rot:])


def test_usual_and_other_calls_are_one():
    """The binding's short way (contiguous tensors, new outputs, the current stream) and its long one (strides, given
    outputs, another stream) give the same, and wrong arguments are refused on either."""
    g = ph.gen(48)
    lens, Hq, Hkv, d, page = [70, 20], 4, 2, 64, 16
    table, total = ph.table_for(g, lens, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, lens)
    length, q = _i32(*lens), ph.randn(g, 2, 1, Hq, d).to(torch.bfloat16)
    usual = blink.blink_paged_token_attention(q, cache, table, length, 70, want_lse=True)
    wide = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    other = blink.blink_paged_token_attention(q, cache, wide[:, :table.shape[1]], length, 70, out=torch.empty_like(q), want_lse=True)
    assert torch.equal(usual[0], other[0]) and torch.equal(usual[1], other[1])
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(length=length.long()), dict(length=length[:1]), dict(table=table.long()),
                dict(table=table[:1]), dict(q=q[..., :32]), dict(ws=torch.zeros(64, device="cuda")), dict(cache={**cache, "v": cache["v"][:1]}),
                dict(cache={**cache, "k_scale": cache["k_scale"].view(torch.uint8)}), dict(q=q.cpu()), dict(q=None), dict(max_len=2**40)):
        a = dict(q=q, cache=cache, table=table, length=length, max_len=70, ws=None)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            blink.blink_paged_token_attention(a["q"], a["cache"], a["table"], a["length"], a["max_len"], ws=a["ws"])
    with pytest.raises(blink.BlinkError):
        blink.blink_paged_token_attention(q, cache, table, length, 131073)
    k = ph.randn(g, 3, Hkv, d).to(torch.bfloat16)
    turns, _ = blink.blink_rope_table(d)
    for bad in (dict(k=k.half()), dict(v=k[:2]), dict(cu=_i32(0, 2)), dict(start=_i32(0)), dict(turns=turns.float()),
                dict(turns=torch.zeros(33, dtype=torch.int64, device="cuda")), dict(ws=torch.zeros(64, device="cuda")), dict(k=k[..., ::2]),
                dict(start=_i32(0, 0).cpu()), dict(positions=_i32(1, 2))):
        a = dict(k=k, v=k, cu=_i32(0, 2, 3), start=_i32(0, 0), turns=turns, ws=None, positions=None)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            blink.blink_paged_append(a["k"], a["v"], cache, table, a["cu"], a["start"], 2, positions=a["positions"], turns=a["turns"], ws=a["ws"])
    rows = ph.randn(g, 5, Hq, d).to(torch.bfloat16)
    kv = ph.randn(g, 5, Hkv, d).to(torch.bfloat16)
    for bad in (dict(q=rows[0]), dict(k=kv[:4]), dict(v=kv.float()), dict(cu=_i32(0, 5, 5)), dict(prefix=[70]), dict(req=[0, 5]),
                dict(cu=_i32(0, 5).cpu()), dict(prefix=[70, 2**33])):
        a = dict(q=rows, k=kv, v=kv, cu=_i32(0, 5), prefix=[70, 20], req=[0, 5, 5])
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            blink.blink_paged_prefix_tail_attention(a["q"], cache, table, a["prefix"], a["k"], a["v"], a["cu"], 1, 5, req_rows=a["req"])
    for bad in (dict(q=rows.half()), dict(k=kv[:4]), dict(pos=_i32(1, 2)), dict(turns=turns.int()), dict(turns=turns[:0]), dict(pos=None)):
        a = dict(q=rows, k=kv, pos=_i32(0, 1, 2, 3, 4), turns=turns)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            blink.blink_rope(a["q"], a["k"], a["pos"], a["turns"])


def test_a_single_row_of_a_projection():
    """One token: slices of one projection's row, whose first stride means nothing."""
    g = ph.gen(49)
    Hq, Hkv, d = 4, 2, 64
    row = ph.randn(g, 1, (Hq + 2 * Hkv) * d).to(torch.bfloat16)
    q, k, v = row[:, :Hq * d].view(1, Hq, d), row[:, Hq * d:(Hq + Hkv) * d].view(1, Hkv, d), row[:, (Hq + Hkv) * d:].view(1, Hkv, d)
    odd = torch.as_strided(k, (1, Hkv, d), (1, d, 1))  # as a single row's stride may be
    turns, _ = blink.blink_rope_table(d)
    qr, kr = blink.blink_rope(q, odd, _i32(77), turns)
    theta, _ = ph.frequencies(d, 10000.0)
    for got, x in ((qr, q), (kr, k)):
        want, size = ph.rotate(x, _i32(77), theta, 1.0, False)
        assert bool(((got.double() - want).abs() <= ph.BF16 * want.abs() + 8 * ph.F32 * size + 2.0 ** -133).all())
    a, b = (blink.blink_paged_cache(2, 16, Hkv, d) for _ in range(2))
    blink.blink_paged_append(odd, v, a, _i32(1).view(1, 1), _i32(0, 1), _i32(5), 1, turns=turns)
    blink.blink_paged_append(k.contiguous(), v.contiguous(), b, _i32(1).view(1, 1), _i32(0, 1), _i32(5), 1, turns=turns)
    assert all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) for n in a)


def test_calls_behind_one_another_see_what_was_written():
    """Rotation, append, token attention and few-row prefix-tail attention issued without a pause, each reading what the
    one before wrote, against the same calls with the device waited for in between."""
    g = ph.gen(50)
    S, Hq, Hkv, d, page, P = 2, 8, 2, 64, 16, 700
    table, total = ph.table_for(g, [P + 64] * S, page)
    filled = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, filled, table, [P] * S)
    turns, _ = blink.blink_rope_table(d)
    n = 30
    x = [tuple(ph.randn(g, S, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv)) for _ in range(n)]
    one = _i32(0, 1, 2)
    starts = [_i32(P + i, P + i) for i in range(n + 1)]
    ws = [blink.new_workspace(1 << 22, "cuda") for _ in range(3)]

    def steps(wait):
        cache = {k: v.clone() for k, v in filled.items()}
        q_buf, k_buf = torch.empty_like(x[0][0]), torch.empty_like(x[0][1])
        torch.cuda.synchronize()
        got = []
        for i, (q, k, v) in enumerate(x):
            blink.blink_rope(q, k, starts[i], turns, q_out=q_buf, k_out=k_buf)
            wait()
            out, lse, _ = blink.blink_paged_prefix_tail_attention(q_buf, cache, table, [P, P + i], k_buf, v, one, 2, 1, req_rows=[0, 1, 2],
                                                                  want_lse=True, ws=ws[0])
            wait()
            blink.blink_paged_append(k, v, cache, table, one, starts[i], 1, turns=turns, ws=ws[1])
            wait()
            tok, lse2, _ = blink.blink_paged_token_attention(q_buf.view(S, 1, Hq, d), cache, table, starts[i + 1], P + n, want_lse=True, ws=ws[2])
            wait()
            got += [out, lse, tok, lse2]
        torch.cuda.synchronize()
        return got
    slow, fast = steps(torch.cuda.synchronize), steps(lambda: None)
    assert all(torch.equal(a, b) for a, b in zip(slow, fast))


def test_captured_behind_copies_and_other_streams():
    """Calls captured right behind a copy, a fill, and work of another stream that is waited for: they see its results."""
    g = ph.gen(51)
    S, Hq, Hkv, d, page, P = 2, 8, 2, 64, 16, 3000
    table, total = ph.table_for(g, [P + 8] * S, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, [P] * S)
    turns, _ = blink.blink_rope_table(d)
    new = [ph.randn(g, S, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv)]
    q, k, v = (torch.zeros_like(x) for x in new)
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    pos, length = _i32(0, 0), _i32(0, 0)
    one = _i32(0, 1, 2)
    ws = [blink.new_workspace(1 << 22, "cuda") for _ in range(3)]
    out, tok = torch.empty_like(q), torch.empty(S, 1, Hq, d, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()

    def work():
        main = torch.cuda.current_stream()
        pos.fill_(P)
        for a, b in zip((q, k, v), new):
            a.copy_(b)                                   # copies
        blink.blink_rope(q, k, pos, turns, q_out=qr, k_out=kr)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            length.copy_(pos)
            length.add_(1)
        blink.blink_paged_append(k, v, cache, table, one, pos, 1, turns=turns, ws=ws[0])
        main.wait_stream(side)                           # two grids, of two streams, before the next call
        blink.blink_paged_token_attention(qr.view(S, 1, Hq, d), cache, table, length, P + 8, out=tok, ws=ws[1])
        out.zero_()
        blink.blink_paged_prefix_tail_attention(qr, cache, table, [P, P], kr, v, one, 2, 1, req_rows=[0, 1, 2], out=out, ws=ws[2])
    work()
    torch.cuda.synchronize()
    want = (out.clone(), tok.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(20):
        for x in (q, k, v, qr, kr, pos, length, out, tok):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(tok, want[1])
    ph.check_attention(tok, blink.blink_paged_token_attention(qr.view(S, 1, Hq, d), cache, table, length, P + 8, want_lse=True)[1],
                       ph.token_reference(qr.view(S, 1, Hq, d), cache, table, [P + 1] * S))


@pytest.mark.parametrize("d,page", [(128, 64), (64, 16)])
def test_pages_never_written_are_zeros(d, page):
    """Lengths that take in pages that nothing was written to: a cache's zeros, with scales of byte 0, between pages whose
    values are large.  Such keys score 0 and add zeros."""
    g = ph.gen(52)
    lens, Hq, Hkv = [900, 77, 2500], 8, 2
    table, total = ph.table_for(g, lens, page)
    cache = blink.blink_paged_cache(total, page, Hkv, d)
    written = [list(range(0, -(-n // page), 2 + s)) for s, n in enumerate(lens)]  # every second, third, fourth page
    for s, n in enumerate(lens):
        for i in written[s]:
            k, v = (0.3 * ph.randn(g, page, Hkv, d).to(torch.bfloat16) for _ in range(2))
            v = v * 2.0 ** (3 * (i % 5) - 2)
            blink.blink_paged_append(k, v, cache, table[s:s + 1, i:i + 1], _i32(0, page), _i32(0), page)
    q = ph.randn(g, 3, 4, Hq, d).to(torch.bfloat16)
    out, lse, ws = blink.blink_paged_token_attention(q, cache, table, _i32(*lens), max(lens), want_lse=True)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    ph.check_attention(out, lse, ph.token_reference(q, cache, table, lens))
    pre = [[ph.values(cache, n, table[s], lens[s]) for n in ("k", "v")] for s in range(3)]
    for r in (1, 90):  # rows of a request: from the pages, and by way of bf16 rows
        rows = 3 * r
        qt, kt, vt = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
        got, got_lse, ws = blink.blink_paged_prefix_tail_attention(qt, cache, table, lens, kt, vt, _i32(0, r, 2 * r, rows), 3, r,
                                                                   req_rows=[0, r, 2 * r, rows], want_lse=True)
        assert blink.blink_read_device_status(ws) == blink.BLINK_OK
        ref = []
        for i in range(rows):
            s = i // r
            k, v = (torch.cat([x, y[s * r:i + 1].double().transpose(0, 1)], dim=1) for x, y in zip(pre[s], (kt, vt)))
            ref.append(ph.attend(qt[i], k, v, 1 / math.sqrt(d)))
        o, l, mag, size = zip(*ref)
        o, l = torch.stack(o)[:, None], torch.stack(l, dim=1)
        if r == 1:
            ph.check_attention(got[:, None], got_lse, (o, l, torch.stack(mag, dim=1)[:, :, None], torch.stack(size, dim=1)))
        else:  # the attention's own tolerances
            assert float((got.double() - o[:, 0]).abs().max()) <= 2e-2 * float(o.abs().max())
            assert float((got_lse.double() - l).abs().max()) <= 2e-3 * max(1.0, float(l.abs().max()))


def test_scales_outside_the_range_are_read_as_the_nearest():
    g = ph.gen(53)
    P, Hq, Hkv, d, page = 500, 4, 2, 64, 32
    table, total = ph.table_for(g, [P], page)
    one = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, one, table, [P], k_exp=(-10, -8))
    two = {n: x.clone() for n, x in one.items()}
    for n, bytes_ in (("k_scale", (0, 1, 60, 78)), ("v_scale", (0, 40, 200, 255, 160, 78))):
        for i, b in enumerate(bytes_):
            one[n].view(torch.uint8)[table[0, 2 * i].long()] = b
            two[n].view(torch.uint8)[table[0, 2 * i].long()] = min(max(b, 127 - 48), 127 + 32)
    q = ph.randn(g, 1, 1, Hq, d).to(torch.bfloat16)
    want, lse, _ = blink.blink_paged_token_attention(q, two, table, _i32(P), P, want_lse=True)
    got, got_lse, _ = blink.blink_paged_token_attention(q, one, table, _i32(P), P, want_lse=True)
    assert torch.equal(got, want) and torch.equal(got_lse, lse)
    ph.check_attention(want, lse, ph.token_reference(q, two, table, [P]))
    for rows in (2, 100):
        qt, kt, vt = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
        a, b = (blink.blink_paged_prefix_tail_attention(qt, c, table, [P], kt, vt, _i32(0, rows), 1, rows)[0] for c in (one, two))
        assert torch.equal(a, b) and bool(a.isfinite().all())


@pytest.mark.parametrize("byte", [0, 50, 255])
def test_append_behind_slots_of_a_page_never_written(byte):
    """A page whose first slots hold zeros with a scale outside the range: the zeros stay, the new tokens get the scale that
    they need (or the largest one, where the page has it)."""
    g = ph.gen(54)
    Hkv, d, page, filled, n = 2, 128, 32, 5, 9
    cache = blink.blink_paged_cache(1, page, Hkv, d)
    for s in ("k_scale", "v_scale"):
        cache[s].view(torch.uint8).fill_(byte)
    k, v = (2000 * ph.randn(g, n, Hkv, d).to(torch.bfloat16) for _ in range(2))
    blink.blink_paged_append(k, v, cache, _i32(0).view(1, 1), _i32(0, n), _i32(filled), n)
    for name, x in (("k", k), ("v", v)):
        codes = cache[name].view(torch.uint8)[0]
        assert bool((codes[:, :filled] == 0).all()) and bool((codes[:, filled + n:] == 0).all())
        for h in range(Hkv):
            e = 32 if byte == 255 else ph.scale_exponent(float(x[:, h].abs().max()))
            assert int(cache[name + "_scale"].view(torch.uint8)[0, h]) == 127 + e
            assert torch.equal(codes[h, filled:filled + n].view(torch.float8_e4m3fn).double(), ph.e4m3(x[:, h].double() * 2.0 ** -e))


@pytest.mark.parametrize("S,page,long_at", [(40, 16, (7,)), (3, 64, (2,)), (200, 32, (0, 150)), (3000, 16, (2999,))])
def test_append_one_long_sequence_among_short_ones(S, page, long_at):
    """max_new far above what most sequences get: the same bits as one call for each kind, rows of a slice (cu does not start
    at 0), empty sequences, and a bad sequence flagged that leaves the others as they should be."""
    g = ph.gen(S)
    Hkv, d = 2, 64
    new = torch.randint(0, 4, (S,), generator=torch.Generator().manual_seed(S)).tolist()
    for i in long_at:
        new[i] = 1000 + i
    start = torch.randint(0, 3 * page, (S,), generator=torch.Generator().manual_seed(S + 1)).tolist()
    ends = [a + b for a, b in zip(start, new)]
    table, total = ph.table_for(g, ends, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, start if S < 300 else [0] * S)
    other = {n: x.clone() for n, x in cache.items()}
    third = {n: x.clone() for n, x in cache.items()}
    n = sum(new)
    k, v = (ph.randn(g, n, Hkv, d).to(torch.bfloat16) for _ in range(2))
    cu = [sum(new[:i]) for i in range(S + 1)]
    turns, _ = blink.blink_rope_table(d)
    most = max(new)
    assert n // page + 2 * S < ((most + page - 2) // page + 1) * S
    ws = blink.blink_paged_append(k, v, cache, table, _i32(*cu) + 5, _i32(*start), most, turns=turns)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    short = [0 if i in long_at else x for i, x in enumerate(new)]
    rows = [r for i in range(S) if i not in long_at for r in range(cu[i], cu[i + 1])]
    cus = [sum(short[:i]) for i in range(S + 1)]
    blink.blink_paged_append(k[rows], v[rows], other, table, _i32(*cus), _i32(*start), 4, turns=turns)
    for i in long_at:
        blink.blink_paged_append(k[cu[i]:cu[i + 1]], v[cu[i]:cu[i + 1]], other, table[i:i + 1], _i32(0, new[i]), _i32(start[i]), new[i], turns=turns)
    for x in cache:
        assert torch.equal(cache[x].view(torch.uint8), other[x].view(torch.uint8))
    # a bad start: flagged, its pages left, the rest written
    bad = next(i for i in range(S) if new[i] and i not in long_at)
    worse = list(start)
    worse[bad] = -1
    ws = blink.blink_paged_append(k, v, third, table, _i32(*cu), _i32(*worse), most, turns=turns)
    assert blink.blink_read_device_status(ws) == blink.BLINK_DEVICE_FLAG
    kept = torch.ones(total, dtype=torch.bool, device="cuda")
    kept[table[bad][table[bad] >= 0].long()] = False
    for x in cache:
        assert torch.equal(cache[x].view(torch.uint8)[kept], third[x].view(torch.uint8)[kept])


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 8), (1, 4, 1), (3, 16, 2)])
@pytest.mark.parametrize("bound", [10000, 131072])
def test_sequences_shorter_than_the_bound(T, Hq, Hkv, bound):
    """Lengths about the borders of how a sequence is cut, one sequence at a time and several."""
    g = ph.gen(T + Hkv + bound)
    d, page = 64, 64
    lens = [1, 63, 64, 65, 1000, 2048, 2049, 3647, 3648, 3649, 7295, 7296, 7297, 9999, 10000]
    table, total = ph.table_for(g, [10000], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, [10000])
    ws = blink.new_workspace(blink.paged_token_attention_workspace_bytes(len(lens), T, bound, Hq, Hkv, d), "cuda")
    q = ph.randn(g, len(lens), T, Hq, d).to(torch.bfloat16)
    for n, x in zip(lens, q):
        out, lse, _ = blink.blink_paged_token_attention(x[None], cache, table, _i32(n), bound, want_lse=True, ws=ws)
        ph.check_attention(out, lse, ph.token_reference(x[None], cache, table, [n]))
    rows = table.expand(len(lens), -1).contiguous()
    out, lse, _ = blink.blink_paged_token_attention(q, cache, rows, _i32(*lens), bound, want_lse=True, ws=ws)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    ph.check_attention(out, lse, ph.token_reference(q, cache, rows, lens))


@pytest.mark.parametrize("S,T,Hq,Hkv,d,page", [(70, 1, 16, 4, 128, 64), (90, 3, 24, 4, 64, 16), (300, 1, 8, 8, 64, 32), (1030, 2, 2, 1, 64, 16),
                                               (40, 4, 16, 4, 128, 64), (1024, 1, 2, 1, 64, 16)])
def test_many_sequences_far_below_the_bound(S, T, Hq, Hkv, d, page):
    """max_len 131072 (a call captured for any length) over many short sequences, some empty, and one long one, over one
    table: the plain form's results, the same bits each time, and bad lengths cut and flagged."""
    g = ph.gen(S + T)
    some = torch.randint(0, 700, (S,), generator=torch.Generator().manual_seed(S)).tolist()
    lens = [0 if i % 11 == 0 else n for i, n in enumerate(some)]
    lens[S - 3], lens[S // 2], lens[1] = 9000, 2049, 1
    row, total = ph.table_for(g, [9000], page)  # the sequences share their pages
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, row, [9000])
    table = row.expand(S, -1).contiguous()
    q = ph.randn(g, S, T, Hq, d).to(torch.bfloat16)
    length = _i32(*lens)
    out, lse, ws = blink.blink_paged_token_attention(q, cache, table, length, 131072, want_lse=True)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    ph.check_attention(out, lse, ph.token_reference(q, cache, table, lens))
    for _ in range(5):
        again, lse2, _ = blink.blink_paged_token_attention(q, cache, table, length, 131072, want_lse=True, ws=ws)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    worse = list(lens)
    worse[0], worse[S - 1] = -7, 131073
    cut = list(lens)
    cut[0], cut[S - 1] = 0, row.shape[1] * page
    if cut[S - 1] > 9000:  # the table's last slots hold no token
        table = table[:, :9000 // page].contiguous()
        cut = [min(n, 9000 // page * page) for n in cut]
        worse = [min(n, 9000 // page * page) if n <= 9000 else n for n in worse]
    out, lse, ws = blink.blink_paged_token_attention(q, cache, table, _i32(*worse), 131072, want_lse=True, ws=ws)
    assert blink.blink_read_device_status(ws) == blink.BLINK_DEVICE_FLAG
    ph.check_attention(out, lse, ph.token_reference(q, cache, table, cut))


def test_two_captured_calls_far_below_the_bound():
    """Two graphs over one workspace, each for many sequences whose lengths change between replays."""
    g = ph.gen(55)
    S, Hq, Hkv, d, page, most = 80, 8, 4, 128, 64, 4000
    row, total = ph.table_for(g, [most], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, row, [most])
    table = row.expand(S, -1).contiguous()
    qs = [ph.randn(g, S, 1, Hq, d).to(torch.bfloat16) for _ in range(2)]
    length, outs, graphs = torch.full((S,), 100, dtype=torch.int32, device="cuda"), [torch.empty_like(qs[0]) for _ in range(2)], []
    ws = blink.new_workspace(blink.paged_token_attention_workspace_bytes(S, 1, 131072, Hq, Hkv, d), "cuda")
    for i in range(2):
        blink.blink_paged_token_attention(qs[i], cache, table, length, 131072, out=outs[i], ws=ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            blink.blink_paged_token_attention(qs[i], cache, table, length, 131072, out=outs[i], ws=ws)
    for step in range(6):
        lens = torch.randint(0, most if step % 2 else 90, (S,), device="cuda", generator=g).to(torch.int32)
        length.copy_(lens)
        for i in (0, 1, 0):
            graphs[i].replay()
        for i in range(2):
            want, _, _ = blink.blink_paged_token_attention(qs[i], cache, table, lens, most)
            a, b = outs[i].double(), want.double()  # cut otherwise: each within half a step and the weights' roundings
            assert float((a - b).abs().max()) <= 2e-2 * float(b.abs().max())
            assert bool((outs[i][lens == 0] == 0).all())
    torch.cuda.synchronize()
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK


@pytest.mark.parametrize("Hq,Hkv,d,page,most", [(4, 2, 64, 16, 12), (4, 4, 128, 64, 3)])
def test_few_tail_rows_against_prefixes_of_unequal_lengths(Hq, Hkv, d, page, most):
    """64 requests of a few rows, or none, against prefixes of 0 to 131072 tokens: one question each."""
    g = ph.gen(most)
    prefix = torch.randint(0, 500, (64,), generator=torch.Generator().manual_seed(most)).tolist()
    prefix[5], prefix[40], prefix[63] = 131072, 0, 5000
    news = torch.randint(0, most + 1, (64,), generator=torch.Generator().manual_seed(most + 1)).tolist()
    news[5], news[40], news[63] = 2, 1, most
    row, total = ph.table_for(g, [131072], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    scale = [torch.randint(119, 123, (total, Hkv), device="cuda", generator=g).to(torch.uint8) for _ in range(2)]
    for n, e in zip("kv", scale):
        cache[n].view(torch.uint8).copy_((110 * ph.randn(g, *cache[n].shape)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        cache[n + "_scale"].view(torch.uint8).copy_(e)
    table = row.expand(64, -1).contiguous()  # requests share their pages
    at = [sum(news[:i]) for i in range(65)]
    cu = sorted(set(at))
    rows = at[-1]
    q, k, v = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    args = (q, cache, table, prefix, k, v, _i32(*cu), len(cu) - 1, most)
    out, lse, ws = blink.blink_paged_prefix_tail_attention(*args, req_rows=at, want_lse=True)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    ref = []
    for r in range(64):
        pre = [ph.values(cache, n, table[r], prefix[r]) for n in "kv"]
        for i in range(at[r], at[r + 1]):
            kk, vv = (torch.cat([x, y[at[r]:i + 1].double().transpose(0, 1)], dim=1) for x, y in zip(pre, (k, v)))
            ref.append(ph.attend(q[i], kk, vv, 1 / math.sqrt(d)))
    o, l, mag, size = zip(*ref)
    ph.check_attention(out[:, None], lse, (torch.stack(o)[:, None], torch.stack(l, dim=1), torch.stack(mag, dim=1)[:, :, None],
                                           torch.stack(size, dim=1)))
    for _ in range(3):
        again, lse2, _ = blink.blink_paged_prefix_tail_attention(*args, req_rows=at, want_lse=True, ws=ws)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
