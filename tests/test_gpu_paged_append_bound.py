"""The append's bound of new tokens where it is zero."""
import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402


@pytest.mark.parametrize("news,flagged", [([0, 0, 0], False), ([0, 2, 0], True), ([1, 1, 1], True)])
def test_a_bound_of_no_tokens_is_checked(news, flagged):
    """max_new 0 with rows of k and v: a sequence with new tokens is longer than the bound, which is flagged, and nothing is
    written; rows behind the last sequence are no sequence's."""
    g = ph.gen(72)
    Hkv, d, page, S = 2, 64, 16, len(news)
    table, total = ph.table_for(g, [20] * S, page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    x = ph.randn(g, 4, Hkv, d).to(torch.bfloat16)
    cu = torch.tensor([sum(news[:i]) for i in range(S + 1)], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 3, 16], dtype=torch.int32, device="cuda")
    before = {n: t.clone() for n, t in cache.items()}
    ws = blink.blink_paged_append(x, x, cache, table, cu, start, 0)
    assert blink.blink_read_device_status(ws) == (blink.BLINK_DEVICE_FLAG if flagged else blink.BLINK_OK)
    assert all(torch.equal(cache[n].view(torch.uint8), before[n].view(torch.uint8)) for n in cache)
