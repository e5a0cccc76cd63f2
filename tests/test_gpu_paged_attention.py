"""Attention of last tokens over the 8-bit pages against the plain form in 64 bits: lengths of none and one, pages that
end inside a step, several tokens, head groups, NaN in slots that nobody sees, far scales, long caches cut into chunks."""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402


def _case(seed, lens, T, Hq, Hkv, d, page, fused=False, k_exp=(-8, -5), v_exp=(-8, -5)):
    g = ph.gen(seed)
    table, total = ph.table_for(g, lens, page)
    cache = ph.new_cache(g, total, Hkv, page, d, fused=fused)
    ph.fill(g, cache, table, lens, k_exp, v_exp)
    q = ph.randn(g, len(lens), T, Hq, d).to(torch.bfloat16)
    return q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def _run(q, cache, table, length, max_len, **kw):
    out, lse, ws = blink.blink_paged_token_attention(q, cache, table, length, max_len, want_lse=True, **kw)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    return out, lse


LENS = [0, 1, 2, 5, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 200, 300]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (32, 8, 128), (5, 1, 64), (40, 2, 128), (8, 8, 128), (17, 1, 64)])
def test_token_attention_lengths(page, T, Hq, Hkv, d):
    """Every slot that no sequence holds is NaN."""
    q, cache, table, length = _case(page + T, LENS, T, Hq, Hkv, d, page, fused=page == 64)
    out, lse = _run(q, cache, table, length, 300)
    ph.check_attention(out, lse, ph.token_reference(q, cache, table, LENS))


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (4, 8, 2), (16, 32, 1), (64, 1, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[9000], [20000, 3, 4097, 12288]])
def test_token_attention_long(T, Hq, Hkv, d, lens):
    q, cache, table, length = _case(T + d, lens, T, Hq, Hkv, d, 128)
    out, lse = _run(q, cache, table, length, max(lens))
    ph.check_attention(out, lse, ph.token_reference(q, cache, table, lens))
    again, lse2 = _run(q, cache, table, length, max(lens))
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_token_attention_longest():
    """131072 tokens, with a larger bound on the other sequence's length than it has."""
    lens = [131072, 77]
    q, cache, table, length = _case(2, lens, 1, 4, 1, 128, 64)
    out, lse = _run(q, cache, table, length, 131072)
    ph.check_attention(out, lse, ph.token_reference(q, cache, table, lens))


@pytest.mark.parametrize("exps", [(-48, -40), (20, 32), (-24, 24)])
@pytest.mark.parametrize("T", [1, 2])
def test_token_attention_value_scales(exps, T):
    """Pages whose values are far apart: the large ones decide, and where a row's weight is on small ones, they do."""
    lens = [400, 33, 1500]
    q, cache, table, length = _case(7, lens, T, 8, 2, 128, 16, v_exp=exps)
    out, lse = _run(q, cache, table, length, 1500)
    ph.check_attention(out, lse, ph.token_reference(q, cache, table, lens))


def test_token_attention_weight_on_small_values():
    """The keys with nearly all the weight have values 2^-20 of the others'."""
    lens, d, page = [256], 64, 16
    q, cache, table, length = _case(3, lens, 1, 4, 1, d, page, k_exp=(-8, -8), v_exp=(8, 8))
    for i in (0, 7, 15):
        p = int(table[0, i])
        cache["v_scale"].view(torch.uint8)[p] = 127 - 12
        cache["k"].view(torch.uint8)[p] = (60.0 * q[0, 0, 0].float()).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        cache["k_scale"].view(torch.uint8)[p] = 127
    q[0, 1:] = q[0, :1]
    out, lse = _run(q, cache, table, length, 256)
    ref = ph.token_reference(q, cache, table, lens)
    ph.check_attention(out, lse, ref)


@pytest.mark.parametrize("size", [1e-20, 1e4, 1e15])
def test_token_attention_large_and_small_queries(size):
    lens = [100, 17]
    q, cache, table, length = _case(5, lens, 1, 4, 2, 64, 32)
    q = (q.float() * size).to(torch.bfloat16)
    q[1, 0, 0] = 0
    out, lse = _run(q, cache, table, length, 100, scale=1e-3 / size)
    ph.check_attention(out, lse, ph.token_reference(q, cache, table, lens, scale=1e-3 / size))


def test_token_attention_rising_and_falling_scores():
    """Scores that rise by hundreds over the keys, and that fall: the running maximum moves often, or never."""
    d, page = 64, 16
    for sign in (1.0, -1.0):
        lens = [500]
        q, cache, table, length = _case(1, lens, 1, 2, 1, d, page)
        q.zero_()
        q[..., 0] = 16.0
        for i in range(-(-500 // page)):
            p = int(table[0, i])
            cache["k"].view(torch.uint8)[p] = 0
            cache["k"].view(torch.uint8)[p, 0, :, 0] = (sign * (torch.arange(page, device="cuda") + page * i).float() / 2 - 120).to(
                torch.float8_e4m3fn).view(torch.uint8)
            cache["k_scale"].view(torch.uint8)[p] = 127
        out, lse = _run(q, cache, table, length, 500)
        ph.check_attention(out, lse, ph.token_reference(q, cache, table, lens))


def test_token_attention_nan_where_it_is_not_seen():
    """A NaN value in the newest token reaches that token alone; a NaN key makes the rows that see it NaN."""
    T, Hq, Hkv, d, page = 4, 4, 2, 64, 16
    lens = [50, 50]
    q, cache, table, length = _case(11, lens, T, Hq, Hkv, d, page)
    clean, lse0 = _run(q, cache, table, length, 50)
    p, slot = int(table[0, 3]), 49 - 48
    cache["v"].view(torch.uint8)[p, 1, slot, 5] = 0x7F
    out, lse = _run(q, cache, table, length, 50)
    assert torch.equal(lse, lse0)
    where = out.isnan()
    assert bool(where[0, 3, 2:, 5].all()) and int(where.sum()) == 2
    assert torch.equal(out[~where], clean[~where])
    cache["v"].view(torch.uint8)[p, 1, slot, 5] = 0x10
    cache["k"].view(torch.uint8)[p, 0, slot, 9] = 0xFF
    out, lse = _run(q, cache, table, length, 50)
    assert bool(out[0, 3, :2].isnan().all()) and bool(lse.view(Hq, 2, T)[:2, 0, 3].isnan().all())
    assert bool(out[0, :3].isfinite().all()) and bool(out[1].isfinite().all()) and bool(out[0, 3, 2:].isfinite().all())


def test_token_attention_nan_and_infinite_queries():
    lens = [5000]
    q, cache, table, length = _case(12, lens, 1, 4, 2, 64, 64)
    clean, _ = _run(q, cache, table, length, 5000)
    q[0, 0, 1, 3] = math.nan
    q[0, 0, 2, 3] = math.inf
    out, lse = _run(q, cache, table, length, 5000)
    assert bool(out[0, 0, 1].isnan().all()) and bool(out[0, 0, 2].isnan().all()) and bool(lse[1:3].isnan().all())
    assert torch.equal(out[0, 0, 0], clean[0, 0, 0]) and torch.equal(out[0, 0, 3], clean[0, 0, 3])


def test_token_attention_bad_pages_and_lengths():
    """A bad page counts as absent, a bad length is cut; both are flagged and the other sequences are right."""
    lens = [100, 100, 60, 100]
    q, cache, table, length = _case(13, lens, 1, 4, 2, 64, 16)
    good = ph.token_reference(q, cache, table, lens)
    bad = table.clone()
    bad[1, 2], bad[1, 5] = cache["k"].shape[0], -7
    length[2], length[3] = -5, 100000
    out, lse, ws = blink.blink_paged_token_attention(q, cache, bad, length, 100, want_lse=True)
    assert blink.blink_read_device_status(ws) == blink.BLINK_DEVICE_FLAG
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    out_ok, lse_ok = out[[0, 3]], lse[:, [0, 3]]
    ph.check_attention(out_ok, lse_ok, (good[0][[0, 3]], good[1][:, [0, 3]], good[2][:, [0, 3]], good[3][:, [0, 3]]))
    assert bool((out[2] == 0).all()) and bool((lse[:, 2] == -math.inf).all())
    k, v = (torch.cat([x[:, :32], x[:, 48:80], x[:, 96:]], dim=1)
            for x in (ph.values(cache, n, table[1], 100) for n in ("k", "v")))
    want = ph.attend(q[1, 0], k, v, 1 / 8)
    assert bool(((out[1, 0].double() - want[0]).abs() <= ph.BF16 * want[0].abs() + 2 * ph.F16 * want[2][0]).all())


def test_token_attention_out_scale_and_streams():
    lens = [1000, 2500]
    q, cache, table, length = _case(14, lens, 2, 8, 2, 128, 64)
    want = ph.token_reference(q, cache, table, lens, scale=0.05)
    out, lse = torch.empty_like(q), torch.empty(8, 4, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, l, ws = blink.blink_paged_token_attention(q, cache, table, length, 2500, scale=0.05, out=out, lse=lse, stream=side)
    assert o is out and l is lse
    side.synchronize()
    ph.check_attention(out, lse, want)
    o2, none, _ = blink.blink_paged_token_attention(q, cache, table, length, 2500, scale=0.05, ws=ws)
    assert none is None and torch.equal(o2, out)
    # a larger bound cuts the work otherwise: the same within the roundings
    o3, l3 = _run(q, cache, table, length, 131072, scale=0.05)
    ph.check_attention(o3, l3, want)


# ---------------------------------------------------------------------------------------------- prefix in pages
def _tail_reference(q, cache, table, prefix, req_rows, k_tail, v_tail, cu, scale):
    rows, Hq, d = q.shape
    out = torch.empty(rows, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(Hq, rows, dtype=torch.float64, device="cuda")
    for b in range(len(cu) - 1):
        r = next(i for i in range(len(prefix)) if req_rows[i] <= cu[b] < req_rows[i + 1])
        P = prefix[r]
        k, v = (ph.values(cache, n, table[r], P) for n in ("k", "v"))
        for i in range(cu[b], cu[b + 1]):
            kk, vv = (torch.cat([x, y[cu[b]:i + 1].double().transpose(0, 1)], dim=1) for x, y in ((k, k_tail), (v, v_tail)))
            out[i], lse[:, i] = ph.attend(q[i], kk, vv, scale)[:2]
    return out, lse


@pytest.mark.parametrize("Hq,Hkv,d,page", [(4, 2, 64, 16), (32, 8, 128, 64), (5, 1, 64, 128), (40, 8, 128, 32)])
@pytest.mark.parametrize("prefix,tails", [([64], [[8, 12, 16, 24]]), ([1], [[1]]), ([300], [[1, 1, 1, 40]]), ([0], [[3, 70]]),
                                          ([129, 500, 0, 33], [[9], [30, 1], [5], [20, 20, 2]]), ([4000], [[2]])])
def test_prefix_tail_in_pages(Hq, Hkv, d, page, prefix, tails):
    """Against the plain form, with NaN in every slot that holds no token of a prefix."""
    g = ph.gen(sum(prefix) + d)
    table, total = ph.table_for(g, prefix, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, prefix)
    flat = [t for r in tails for t in r]
    cu = [sum(flat[:i]) for i in range(len(flat) + 1)]
    req_rows = [sum(sum(r) for r in tails[:i]) for i in range(len(tails) + 1)]
    rows = cu[-1]
    q, k, v = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    out, lse, ws = blink.blink_paged_prefix_tail_attention(q, cache, table, prefix, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                                           len(flat), max(flat), req_rows=req_rows, want_lse=True)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    want, want_lse = _tail_reference(q, cache, table, prefix, req_rows, k, v, cu, 1 / math.sqrt(d))
    # the attention's own tolerances: 2e-2 of the largest output, 2e-3 of the log-sum-exp
    assert float((out.double() - want).abs().max()) <= 2e-2 * float(want.abs().max())
    assert float((lse.double() - want_lse).abs().max()) <= 2e-3 * max(1.0, float(want_lse.abs().max()))


@pytest.mark.parametrize("Hq,Hkv,d,page", [(4, 2, 64, 16), (32, 8, 128, 64), (5, 1, 64, 128), (40, 2, 128, 32), (64, 1, 64, 64)])
@pytest.mark.parametrize("prefix,tails", [([300], [[1]]), ([0], [[1]]), ([9000], [[1, 1, 2]]), ([129, 0, 4000, 33], [[1], [1], [2, 1], [1, 1]]),
                                          ([131072], [[1]]), ([77], [[1] * 3])])
def test_few_tail_rows(Hq, Hkv, d, page, prefix, tails):
    """One token, or a few rows, of each request: closer than the tensor-core form, as no score is rounded and weights
    enter the products in fp16 (the prefix) and 32 bits (the tail).  Slots that hold no token are NaN, in the padding
    rows of k_tail too."""
    g = ph.gen(sum(prefix) + Hq)
    table, total = ph.table_for(g, prefix, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, prefix)
    flat = [t for r in tails for t in r]
    cu = [sum(flat[:i]) for i in range(len(flat) + 1)]
    req_rows = [sum(sum(r) for r in tails[:i]) for i in range(len(tails) + 1)]
    rows = cu[-1]
    q, k, v = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    out, lse, ws = blink.blink_paged_prefix_tail_attention(q, cache, table, prefix, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                                           len(flat), max(flat), req_rows=req_rows, want_lse=True)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    ref = [torch.empty(rows, 1, Hq, d, dtype=torch.float64, device="cuda"), torch.empty(Hq, rows, dtype=torch.float64, device="cuda"),
           torch.empty(2, rows, 1, Hq, d, dtype=torch.float64, device="cuda"), torch.empty(Hq, rows, dtype=torch.float64, device="cuda")]
    for b in range(len(flat)):
        r = next(i for i in range(len(prefix)) if req_rows[i] <= cu[b] < req_rows[i + 1])
        pre = [ph.values(cache, n, table[r], prefix[r]) for n in ("k", "v")]
        for i in range(cu[b], cu[b + 1]):
            kk, vv = (torch.cat([x, y[cu[b]:i + 1].double().transpose(0, 1)], dim=1) for x, y in zip(pre, (k, v)))
            ref[0][i, 0], ref[1][:, i], ref[2][:, i, 0], ref[3][:, i] = ph.attend(q[i], kk, vv, 1 / math.sqrt(d))
    if max(b - a for a, b in zip(req_rows, req_rows[1:])) * (Hq // Hkv) > 64:  # four rows of 20 heads: the tensor-core form,
        # whose weights are rounded to bf16 (half a step 2^-8, against 2^-11)
        assert float((out.double() - ref[0][:, 0]).abs().max()) <= 2e-2 * float(ref[0].abs().max())
        return
    ph.check_attention(out.view(rows, 1, Hq, d), lse, ref)


def test_few_tail_rows_padded_and_bad_questions():
    """Rows of no question get zeros and -inf; a question of a bad length is flagged and the others are right."""
    g = ph.gen(23)
    Hq, Hkv, d, page, P = 4, 2, 64, 16, 100
    table, total = ph.table_for(g, [P], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, [P])
    rows = 12
    q, k, v = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse, ws = blink.blink_paged_prefix_tail_attention(q, cache, table, [P], k, v, i32(5, 7, 12), 2, 5, seq_start=i32(1, 6), want_lse=True)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    none = [0, 3, 4, 5, 11]
    assert bool((out[none] == 0).all()) and bool((lse[:, none] == -math.inf).all())
    want, want_lse = _tail_reference(q[1:3], cache, table, [P], [0, 2], k[1:3], v[1:3], [0, 2], 1 / 8)
    assert float((out[1:3].double() - want).abs().max()) <= 2 * ph.BF16 * float(want.abs().max())
    assert float((lse[:, 1:3].double() - want_lse).abs().max()) <= 1e-5
    # lengths beyond max_tail, none, past the rows; a question that begins before its request's rows
    for cu, B, max_tail, req in ((i32(0, 6, 12), 2, 5, None), (i32(0, 0, 12), 2, 12, None), (i32(0, 13), 1, 13, None),
                                 (i32(0, 8, 12), 2, 8, [0, 4, 12])):
        n = 1 if req is None else 2
        t = table.expand(n, -1).contiguous()
        _, _, ws = blink.blink_paged_prefix_tail_attention(q, cache, t, [P] * n, k, v, cu, B, max_tail, req_rows=req)
        assert blink.blink_read_device_status(ws) == blink.BLINK_DEVICE_FLAG
    bad = table.clone()
    bad[0, 2] = total
    _, _, ws = blink.blink_paged_prefix_tail_attention(q, cache, bad, [P], k, v, i32(0, 12), 1, 12)
    assert blink.blink_read_device_status(ws) == blink.BLINK_DEVICE_FLAG


def test_prefix_tail_forms_agree():
    """The rows of a question alone (the few-row form) and among many others (the tensor-core form)."""
    g = ph.gen(24)
    Hq, Hkv, d, page, P = 32, 8, 128, 64, 777
    table, total = ph.table_for(g, [P], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, [P])
    rows = 3 + 120
    q, k, v = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    many, lse, _ = blink.blink_paged_prefix_tail_attention(q, cache, table, [P], k, v, i32(0, 3, rows), 2, 120, want_lse=True)
    few, lse3, _ = blink.blink_paged_prefix_tail_attention(q[:3], cache, table, [P], k[:3], v[:3], i32(0, 3), 1, 3, want_lse=True)
    assert float((few.double() - many[:3].double()).abs().max()) <= 2e-2 * float(many[:3].abs().max())
    assert float((lse3 - lse[:, :3]).abs().max()) <= 2e-3


def test_prefix_tail_equals_the_arena():
    """Bit for bit what the bf16 arena with the same values gives, for one request and for several that share pages."""
    g = ph.gen(21)
    Hq, Hkv, d, page, P = 32, 8, 128, 64, 1000
    table, total = ph.table_for(g, [P], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, [P])
    k_pre, v_pre = (ph.values(cache, n, table[0], P).transpose(0, 1).to(torch.bfloat16).contiguous() for n in ("k", "v"))
    rows = 90
    q, k, v = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    cu = torch.tensor([0, 30, 31, 90], dtype=torch.int32, device="cuda")
    want, want_lse, _ = blink.blink_prefix_tail_attention(q, k_pre, v_pre, k, v, cu, 3, P, 59, want_lse=True)
    out, lse, _ = blink.blink_paged_prefix_tail_attention(q, cache, table, [P], k, v, cu, 3, 59, want_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    two = table.expand(2, -1).contiguous()
    want, _, _ = blink.blink_prefix_tail_attention_multi(q, k_pre, v_pre, k, v, cu, 3, [0, 31, 90], [0, 0], [P, P - 77], 59)
    out, _, ws = blink.blink_paged_prefix_tail_attention(q, cache, two, [P, P - 77], k, v, cu, 3, 59, req_rows=[0, 31, 90])
    assert torch.equal(out, want)
    bad = two.clone()
    bad[1, 3] = -1
    _, _, ws = blink.blink_paged_prefix_tail_attention(q, cache, bad, [P, P - 77], k, v, cu, 3, 59, req_rows=[0, 31, 90], ws=ws)
    assert blink.blink_read_device_status(ws) == blink.BLINK_DEVICE_FLAG


def test_prefix_tail_padded_layout():
    g = ph.gen(22)
    Hq, Hkv, d, page, P = 4, 2, 64, 32, 130
    table, total = ph.table_for(g, [P], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, [P])
    rows = 40
    q, k, v = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    cu = torch.tensor([0, 7, 20], dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    out, lse, _ = blink.blink_paged_prefix_tail_attention(q, cache, table, [P], k, v, cu, 2, 20, seq_start=seq, want_lse=True)
    k_pre, v_pre = (ph.values(cache, n, table[0], P).transpose(0, 1).to(torch.bfloat16).contiguous() for n in ("k", "v"))
    want, want_lse, _ = blink.blink_prefix_tail_attention(q, k_pre, v_pre, k, v, cu, 2, P, 20, seq_start=seq, want_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert bool((out[7:20] == 0).all()) and bool((lse[:, 33:] == -math.inf).all())
