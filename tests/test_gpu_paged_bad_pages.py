"""Prefix-tail attention over a page table with bad indexes: the outputs, on both ways that a call can take."""
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402


@pytest.mark.parametrize("Hq,Hkv,d,page", [(4, 2, 64, 16), (8, 1, 128, 64)])
@pytest.mark.parametrize("rows", [1, 7, 150])
def test_keys_of_a_bad_page_are_zeros(Hq, Hkv, d, page, rows):
    """Few rows (read from the pages) and many (by way of bf16 rows): a page outside the cache holds keys and values of zero,
    its keys weigh as such, and the call is flagged.  One of the bad pages is the last, not full one."""
    g = ph.gen(page + rows)
    P = 20 * page - 5
    table, total = ph.table_for(g, [P], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, [P])
    bad = table.clone()
    bad[0, 3], bad[0, 11], bad[0, 12], bad[0, 19] = -1, total, 1 << 30, -(1 << 31)
    k, v = (ph.values(cache, n, table[0], P) for n in "kv")
    for i in (3, 11, 12, 19):
        k[:, i * page:(i + 1) * page] = 0
        v[:, i * page:(i + 1) * page] = 0
    q, kt, vt = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    cu = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    out, lse, ws = blink.blink_paged_prefix_tail_attention(q, cache, bad, [P], kt, vt, cu, 1, rows, want_lse=True)
    assert blink.blink_read_device_status(ws) == blink.BLINK_DEVICE_FLAG
    ref = [ph.attend(q[i], *(torch.cat([x, y[:i + 1].double().transpose(0, 1)], dim=1) for x, y in ((k, kt), (v, vt))), 1 / math.sqrt(d))
           for i in range(rows)]
    o, l, mag, size = zip(*ref)
    o, l = torch.stack(o), torch.stack(l, dim=1)
    if rows * Hq // Hkv <= 64:
        ph.check_attention(out[:, None], lse, (o[:, None], l, torch.stack(mag, dim=1)[:, :, None], torch.stack(size, dim=1)))
    else:  # the attention's own tolerances
        assert float((out.double() - o).abs().max()) <= 2e-2 * float(o.abs().max())
        assert float((lse.double() - l).abs().max()) <= 2e-3 * max(1.0, float(l.abs().max()))
