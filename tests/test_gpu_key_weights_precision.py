"""Precision of the key weights against 64 bits, with a bound of each weight's own.

A term is 2^(c s - b) with c = scale log2(e) and b = lse log2(e).  The product s takes d / 16 steps, each of which
cuts off at most 2^-22 of the sum it leaves (one unit in the last place for the result and one for the
products, which are aligned to it).  c and b are each off by two roundings and the difference by one, and
exp2 by 2^-22.  A thread adds one term of every column tile, 5 steps join a warp, 3 the warps, and pieces of
the tiles may be added apart: each addition is to nearest.
"""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("rows,P,Hq,Hkv,d", [
    (1, 600, 32, 8, 128), (1, 600, 4, 2, 64), (8, 600, 8, 2, 128), (30, 600, 8, 2, 64), (12, 600, 40, 8, 128),
    (300, 600, 28, 4, 128), (300, 2050, 16, 2, 64), (1275, 600, 32, 8, 128), (1275, 600, 32, 8, 64)])
@pytest.mark.parametrize("decay", [0.0, 0.5])
def test_weights(rows, P, Hq, Hkv, d, decay):
    g = torch.Generator(device="cuda").manual_seed(rows + d)
    grp = Hq // Hkv
    q = torch.randn(rows, Hq, d, device="cuda", generator=g).to(BF)
    k = torch.randn(P, Hkv, d, device="cuda", generator=g).to(BF)
    qd = q.double().view(rows, Hkv, grp, d).permute(1, 2, 0, 3).reshape(Hkv, grp * rows, d)
    kd = k.double().permute(1, 2, 0)  # [Hkv, d, P]
    scale = 1 / math.sqrt(d)
    s = torch.zeros(Hkv, grp * rows, P, dtype=torch.float64, device="cuda")
    steps = torch.zeros_like(s)
    for a in range(0, d, 16):
        s += torch.bmm(qd[:, :, a:a + 16], kd[:, a:a + 16])
        steps += s.abs()
    lse = torch.logsumexp(scale * s, -1).view(Hq, rows).float() + 0.05
    prev = torch.rand(Hkv, P, device="cuda", generator=g)
    ld = lse.double().view(Hkv, grp * rows, 1)
    x = scale * s - ld
    off = scale * 2.0**-22 * steps + 2.0**-24 * (2 * (scale * s).abs() + 2 * ld.abs() + x.abs()) + 2.0**-22
    adds = 2 * (-(-rows // min(rows, 128 // grp))) + 16
    want = x.exp().sum(1)
    tol = (x.exp() * off).sum(1) * 1.001 + 2.0**-24 * adds * want
    if decay:
        want = want + decay * prev.double()
        tol = tol + 2.0**-24 * want
    w, _ = blink.blink_prefix_key_weights(q, k, lse, prev=prev, decay=decay)
    err = (w.double() - want).abs()
    assert bool((err <= tol).all()), (float((err / want).max()), float((tol / want).max()))
