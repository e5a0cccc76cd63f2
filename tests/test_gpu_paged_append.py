"""Appending to the 8-bit paged cache against the plain form in 64 bits: page and head sizes, rotations, ragged and
empty sequences, pages that fill in several calls, infinities and NaN, what is left as it was, bad pages."""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402


def _reference(cache, table, x, size, name, starts, news):
    """What the cache holds after the call: codes as values before their last rounding (64 bits), what 32-bit roundings
    may move them by, and scales."""
    page = cache[name].shape[2]
    codes = cache[name].double()
    slack = torch.zeros_like(codes)
    scale = cache[name + "_scale"].view(torch.uint8).clone()
    row = 0
    for s, (start, n) in enumerate(zip(starts, news)):
        at = start
        while at < start + n:
            p, o = int(table[s, at // page]), at % page
            m = min(page - o, start + n - at)
            for h in range(x.shape[1]):
                y, z = x[row:row + m, h], size[row:row + m, h]
                fin = y.abs()[y.isfinite()]
                e = ph.scale_exponent(float(fin.max()) if fin.numel() else 0.0)
                if o:
                    old = int(scale[p, h]) - 127
                    e = max(e, old)
                    codes[p, h, :o] = ph.e4m3(codes[p, h, :o] * 2.0 ** (old - e))
                scale[p, h] = e + 127
                codes[p, h, o:o + m] = y / 2.0 ** e
                slack[p, h, o:o + m] = 8 * ph.F32 * z / 2.0 ** e
            row, at = row + m, at + m
    return codes, slack, scale


def _same(cache, name, want, exact):
    codes, slack, scale = want
    assert torch.equal(cache[name + "_scale"].view(torch.uint8), scale)
    got = cache[name].double()
    assert torch.equal(got.isnan(), codes.isnan())
    if exact:
        assert torch.equal(got.nan_to_num(), ph.e4m3(codes).nan_to_num())
    live = ~codes.isnan()
    c = codes.clamp(-448, 448)
    bound = torch.maximum(ph.E4M3 * c.abs(), torch.full_like(c, 2.0 ** -10)) + slack  # half a step; of the subnormal ones 2^-10
    assert bool(((got - c).abs() <= bound)[live].all())


def _clone(cache):
    return {k: v.clone() for k, v in cache.items()}


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,d,rot,interleaved", [(8, 128, 128, False), (2, 64, 64, True), (1, 64, 32, False), (5, 64, 22, False),
                                                   (3, 128, 36, True), (2, 128, 0, False), (2, 128, 2, False)])
def test_append_ragged(page, Hkv, d, rot, interleaved):
    g = ph.gen(page + d + rot)
    starts, news = [0, 0, 5, 64, 100, 15, 130, 7], [1, 200, 3, 64, 29, 0, 1, 121]
    n = sum(news)
    table, total = ph.table_for(g, [a + b for a, b in zip(starts, news)], page)
    cache = ph.new_cache(g, total, Hkv, page, d, fused=page == 32, filler=0x31)
    ph.fill(g, cache, table, starts, k_exp=(-9, -4), v_exp=(-9, -4))
    before = _clone(cache)
    wide = 2 * Hkv * d + 16
    kv = ph.randn(g, n, wide) * torch.exp(ph.randn(g, n, 1))
    kv = kv.to(torch.bfloat16)
    k, v = kv[:, :Hkv * d].view(n, Hkv, d), kv[:, Hkv * d:2 * Hkv * d].view(n, Hkv, d)
    cu = torch.tensor([sum(news[:i]) + 11 for i in range(len(news) + 1)], dtype=torch.int32, device="cuda")
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    turns, amplitude = (blink.blink_rope_table(rot, 500000.0, scaling="by_dim" if rot > 2 else None, factor=4.0, original=4096)
                        if rot else (None, 1.0))
    theta, amp = ph.frequencies(rot, 500000.0, "by_dim" if rot > 2 else None, 4.0, 4096, 1.0, 32.0) if rot else ([], 1.0)
    ws = blink.blink_paged_append(k, v, cache, table, cu, start, max(news), turns=turns, interleaved=interleaved, amplitude=amplitude)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(starts, news)]).cuda()
    kr, size = ph.rotate(k, pos, theta, amp, interleaved) if rot else (k.double(), k.double().abs() * 0)
    _same(cache, "k", _reference(before, table, kr, size, "k", starts, news), exact=not rot)
    vd = v.double()
    _same(cache, "v", _reference(before, table, vd, vd * 0, "v", starts, news), exact=True)
    # the same call again changes nothing, and explicit positions give the same
    once = _clone(cache)
    blink.blink_paged_append(k, v, cache, table, cu, start, max(news) + 40, positions=pos.to(torch.int32), turns=turns,
                             interleaved=interleaved, amplitude=amplitude, ws=ws)
    for x in cache:
        assert torch.equal(cache[x].view(torch.uint8), once[x].view(torch.uint8))


def test_append_explicit_positions():
    g = ph.gen(3)
    n, Hkv, d, page = 40, 2, 64, 16
    table, total = ph.table_for(g, [n], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    k, v = (ph.randn(g, n, Hkv, d).to(torch.bfloat16) for _ in range(2))
    pos = torch.randint(-1000, 131072, (n,), device="cuda", generator=g).to(torch.int32)
    cu, start = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    before = _clone(cache)
    turns, _ = blink.blink_rope_table(d)
    blink.blink_paged_append(k, v, cache, table, cu, start, n, positions=pos, turns=turns)
    kr, size = ph.rotate(k, pos, ph.frequencies(d, 10000.0)[0], 1.0, False)
    _same(cache, "k", _reference(before, table, kr, size, "k", [0], [n]), exact=False)


@pytest.mark.parametrize("page", [16, 128])
def test_append_token_by_token(page):
    """A page that fills one token at a time, its scale growing on the way; two sequences with pages of their own."""
    g = ph.gen(page)
    Hkv, d, S, n = 3, 64, 2, 35
    table, total = ph.table_for(g, [n] * S, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    one = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    want = {x: t for x, t in _clone(cache).items()}
    for t in range(n):
        # every few tokens one is far larger than those before
        big = 2.0 ** (3 * (t // 5) - 12)
        k, v = ((big * ph.randn(g, S, Hkv, d)).to(torch.bfloat16) for _ in range(2))
        blink.blink_paged_append(k, v, cache, table, one, torch.full((S,), t, dtype=torch.int32, device="cuda"), 1)
        for name, x in (("k", k), ("v", v)):
            codes, _, scale = _reference(want, table, x.double(), x.double() * 0, name, [t] * S, [1] * S)
            want[name] = ph.e4m3(codes).to(torch.float8_e4m3fn)
            want[name + "_scale"] = scale.view(torch.float8_e8m0fnu)
            assert torch.equal(cache[name + "_scale"].view(torch.uint8), scale)
            assert torch.equal(cache[name].double().nan_to_num(), want[name].double().nan_to_num())


def test_append_scale_borders():
    """Largest magnitudes at and next to 448 * 2^e, zeros, the smallest and the largest there are."""
    values = [0.0, 448.0, 447.0, 449.0, 450.0, 896.0, 0.875, 0.8789, 1.0, 3.5, 3.52, 2.0 ** -133, 2.0 ** -40, 448 * 2.0 ** -48,
              450 * 2.0 ** -48, 440 * 2.0 ** -48, 2.0 ** -58, 448 * 2.0 ** 32, 464 * 2.0 ** 32, 1e30, 3.38e38]
    S, Hkv, d, page = len(values), 1, 64, 16
    g = ph.gen(9)
    table, total = ph.table_for(g, [1] * S, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    x = torch.zeros(S, Hkv, d, device="cuda")
    for i, m in enumerate(values):
        x[i] = m * torch.rand(Hkv, d, device="cuda", generator=g)
        x[i, 0, 7] = -m
    x = x.to(torch.bfloat16)
    cu, start = torch.arange(S + 1, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    before = _clone(cache)
    blink.blink_paged_append(x, x, cache, table, cu, start, 1)
    for name in ("k", "v"):
        want = _reference(before, table, x.double(), x.double() * 0, name, [0] * S, [1] * S)
        assert torch.equal(cache[name + "_scale"].view(torch.uint8), want[2])
        assert torch.equal(cache[name].double().nan_to_num(), ph.e4m3(want[0]).nan_to_num())


def test_append_infinities_and_nan():
    """The scale is that of the finite values; an infinity takes the largest code, a NaN stays one, and neither
    touches other heads or pages."""
    g = ph.gen(4)
    n, Hkv, d, page = 40, 3, 64, 16
    table, total = ph.table_for(g, [n], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    x = ph.randn(g, n, Hkv, d).to(torch.bfloat16)
    x[3, 1, 5], x[4, 1, 6], x[20, 0, 0], x[39] = math.inf, -math.inf, math.nan, math.inf
    cu, start = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    before = _clone(cache)
    blink.blink_paged_append(x, x, cache, table, cu, start, n)
    for name in ("k", "v"):
        want = _reference(before, table, x.double(), x.double() * 0, name, [0], [n])
        assert torch.equal(cache[name + "_scale"].view(torch.uint8), want[2])
        got = cache[name].double()
        assert torch.equal(got.isnan(), want[0].isnan())
        assert torch.equal(got.nan_to_num(), ph.e4m3(want[0]).nan_to_num())


def test_append_bad_pages_and_lengths():
    """Bad lengths and page indexes are flagged and skipped; the other sequences are written."""
    g = ph.gen(6)
    Hkv, d, page, S = 2, 64, 16, 6
    table, total = ph.table_for(g, [20] * S, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    x = ph.randn(g, 10 * S, Hkv, d).to(torch.bfloat16)
    cu = torch.arange(0, 10 * S + 1, 10, dtype=torch.int32, device="cuda")
    start = torch.zeros(S, dtype=torch.int32, device="cuda")
    good = _clone(cache)
    blink.blink_paged_append(x[50:], x[50:], good, table[5:], torch.tensor([0, 10], dtype=torch.int32, device="cuda"), start[5:], 10)
    bad_table = table.clone()
    bad_table[0, 0], bad_table[1, 0] = total, -1
    start[2], start[3] = -4, 100  # 100: past the table
    cu_bad = cu.clone()
    ws = blink.blink_paged_append(x, x, cache, bad_table, cu_bad, start, 10)
    assert blink.blink_read_device_status(ws) == blink.BLINK_DEVICE_FLAG
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    p4, p5 = int(table[4, 0]), int(table[5, 0])
    for name in cache:
        got, want = cache[name].view(torch.uint8), good[name].view(torch.uint8)
        assert torch.equal(got[p5], want[p5])
        others = [i for i in range(total) if i not in (p4, p5)]
        assert torch.equal(got[others], want[others])  # as they were
    # more new tokens than max_new: nothing of that sequence is written
    fresh = ph.new_cache(g, total, Hkv, page, d)
    ws = blink.blink_paged_append(x, x, fresh, table, cu, torch.zeros_like(start), 9)
    assert blink.blink_read_device_status(ws) == blink.BLINK_DEVICE_FLAG
    assert bool((fresh["k"].view(torch.uint8) == 0x7F).all())


def test_append_another_stream():
    g = ph.gen(8)
    n, Hkv, d, page = 100, 2, 128, 32
    table, total = ph.table_for(g, [n], page)
    x = ph.randn(g, n, Hkv, d).to(torch.bfloat16)
    cu, start = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = ph.new_cache(g, total, Hkv, page, d), ph.new_cache(g, total, Hkv, page, d)
    blink.blink_paged_append(x, x, a, table, cu, start, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    blink.blink_paged_append(x, x, b, table, cu, start, n, stream=side)
    side.synchronize()
    assert all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)
