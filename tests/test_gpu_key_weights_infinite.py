"""Key weights of keys that hold infinities or NaN: what the formula gives, for that key alone, however the rows
fill a tile (rows past the last and columns that no row has are zeros, and zero times infinity is NaN)."""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
INF = float("inf")


@pytest.mark.parametrize("rows,Hq,Hkv,d", [
    (1, 1, 1, 64), (1, 32, 8, 128), (3, 8, 1, 128), (8, 8, 2, 128),  # at most 32 columns
    (9, 8, 2, 128), (20, 10, 2, 64), (16, 7, 1, 128), (64, 4, 2, 64),  # one tile, full and not
    (33, 8, 2, 64), (70, 10, 2, 128), (300, 28, 4, 64), (65, 2, 2, 128), (2, 127, 1, 64)])  # several
@pytest.mark.parametrize("decay", [0.0, 0.5])
def test_infinite_and_nan_keys(rows, Hq, Hkv, d, decay):
    P = 300
    g = torch.Generator(device="cuda").manual_seed(rows + Hq)
    q = torch.randn(rows, Hq, d, device="cuda", generator=g).to(BF)
    q[:, :, 5] = -q[:, :, 5].abs() - 0.25  # every query is below zero there
    k = torch.randn(P, Hkv, d, device="cuda", generator=g).to(BF)
    s = torch.einsum("thgd,phd->hgtp", q.double().view(rows, Hkv, Hq // Hkv, d), k.double()) / math.sqrt(d)
    lse = torch.logsumexp(s, -1).view(Hq, rows).float()
    dead = torch.zeros(rows, dtype=torch.bool, device="cuda")
    if rows > 2:
        dead[rows // 2] = True
        lse[:, dead] = -INF
    prev = torch.rand(Hkv, P, device="cuda", generator=g)
    want, _ = blink.blink_prefix_key_weights(q, k, lse, prev=prev, decay=decay)
    want = want.clone()
    for key, value, weight in ((0, INF, 0.0), (131, -INF, INF), (299, float("nan"), float("nan")), (257, INF, 0.0)):
        k[key, :, 5] = value
        want[:, key] = weight + decay * prev[:, key]
    got, ws = blink.blink_prefix_key_weights(q, k, lse, prev=prev, decay=decay)
    assert torch.equal(got.isnan(), want.isnan())
    num = ~want.isnan()
    assert torch.equal(got[num], want[num])  # a key's weight does not depend on the others
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
    lse[:] = -INF
    w, _ = blink.blink_prefix_key_weights(q, k, lse)
    assert bool((w == 0).all())  # rows that no question owns add nothing, whatever the keys are
