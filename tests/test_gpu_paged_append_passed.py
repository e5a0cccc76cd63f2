"""Appends that turn part of a head, where the values that pass hold what random ones never do."""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402

PARTS = [(128, 64, False), (64, 32, False), (128, 36, True), (64, 22, False), (128, 2, False), (64, 2, True)]


def _append(x, d, rot, interleaved, page=32):
    """(codes of the passed channels [n, Hkv, d - rot], what they should be as bytes) of keys x [n, Hkv, d]; the table of
    frequencies lies within larger ones, which would show in a code that used them."""
    n, Hkv, _ = x.shape
    table, total = ph.table_for(ph.gen(n), [n], page)
    cache = ph.new_cache(ph.gen(n), total, Hkv, page, d)
    inside = torch.full((4 * d,), 0x2123456789ABCDEF, dtype=torch.int64, device="cuda")
    turns = inside[d:d + rot // 2]
    turns.copy_(blink.blink_rope_table(rot)[0])
    cu, start = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = blink.blink_paged_append(x, x, cache, table, cu, start, n, turns=turns, interleaved=interleaved)
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    i = torch.arange(n, device="cuda")
    at = table[0, i // page].long()
    got = cache["k"].view(torch.uint8)[at, :, i % page][..., rot:]
    e = cache["k_scale"].view(torch.uint8)[at].double() - 127
    want = (x[..., rot:].double() * torch.exp2(-e)[..., None]).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    # the values are themselves the nearest codes, and the values that turn are those of the rotation
    values = x[..., rot:].double() * torch.exp2(-e)[..., None]
    assert torch.equal(want.double().nan_to_num(), ph.e4m3(values).nan_to_num())
    y, size = ph.rotate(x, i, ph.frequencies(rot, 10000.0)[0], 1.0, interleaved)
    turned = cache["k"].view(torch.uint8)[at, :, i % page][..., :rot].view(torch.float8_e4m3fn).double()
    c = (y * torch.exp2(-e)[..., None])[..., :rot]
    assert torch.equal(turned.isnan(), c.isnan())
    bound = torch.maximum(ph.E4M3 * c.abs(), torch.full_like(c, 2.0 ** -10)) + 8 * ph.F32 * (size * torch.exp2(-e)[..., None])[..., :rot]
    fine = c.abs() <= 448
    assert bool(((turned - c).abs() <= bound)[fine].all())
    return got, want


@pytest.mark.parametrize("d,rot,interleaved", PARTS)
def test_zeros_of_either_sign_pass(d, rot, interleaved):
    """Passed values of -0 and +0 between others keep their signs, as they do in a call that turns nothing."""
    g = ph.gen(d + rot)
    n, Hkv = 70, 3
    x = ph.randn(g, n, Hkv, d)
    pick = torch.randint(0, 4, x.shape, device="cuda", generator=g)
    x = torch.where(pick == 0, torch.full_like(x, -0.0), torch.where(pick == 1, torch.zeros_like(x), x)).to(torch.bfloat16)
    x[3, 1, rot:] = -0.0
    got, want = _append(x, d, rot, interleaved)
    assert torch.equal(got, want.view(torch.uint8))


@pytest.mark.parametrize("d,rot,interleaved", PARTS)
def test_nan_passes_alone(d, rot, interleaved):
    """A NaN among the passed values is one NaN code: the other values of its key, its pair's place among them, get their own."""
    g = ph.gen(d + rot + 1)
    n, Hkv = 70, 2
    x = ph.randn(g, n, Hkv, d).to(torch.bfloat16)
    alone = torch.rand(n, Hkv, d - rot, device="cuda", generator=g) < 0.1
    x[..., rot:][alone] = math.nan
    got, want = _append(x, d, rot, interleaved)
    assert torch.equal(got.view(torch.float8_e4m3fn).double().isnan(), alone)
    assert torch.equal(got[~alone], want.view(torch.uint8)[~alone])


@pytest.mark.parametrize("d,rot,interleaved", PARTS)
def test_infinities_pass_alone(d, rot, interleaved):
    """Infinities, a NaN and zeros of either sign among the passed values: infinities take the largest code, the scale is that
    of the finite values, and the others get the codes that they have without them."""
    g = ph.gen(d + rot + 2)
    n, Hkv = 70, 2
    x = ph.randn(g, n, Hkv, d).to(torch.bfloat16)
    pick = torch.randint(0, 40, (n, Hkv, d - rot), device="cuda", generator=g)
    for i, value in enumerate((math.inf, -math.inf, math.nan, -0.0, 0.0)):
        x[..., rot:][pick == i] = value
    got, want = _append(x, d, rot, interleaved)
    assert bool((got[pick == 0] == 0x7E).all()) and bool((got[pick == 1] == 0xFE).all())
    assert torch.equal(got[pick != 2], want.view(torch.uint8)[pick != 2])
    assert bool(got[pick == 2].view(torch.float8_e4m3fn).double().isnan().all())
