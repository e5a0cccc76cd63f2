"""Appending keys of zeros (padded rows, pruned channels), whose values are turned like any others."""
import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402


def _median_us(call, calls=10, times=15):
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            call()
    graph.replay()
    took = []
    for _ in range(times):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        took.append(a.elapsed_time(b) * 1e3 / calls)
    return sorted(took)[times // 2]


@pytest.mark.parametrize("interleaved", [False, True])
def test_keys_of_zeros_take_no_longer(interleaved):
    """Every code is a zero, and the call takes about what it takes on random keys: no value of a zero pair is computed
    again.  (Each of them again is 4.8 times the time; half again leaves room for what else runs.)"""
    g = ph.gen(73)
    n, Hkv, d, page = 18432, 8, 128, 64
    table, total = ph.table_for(g, [n], page)
    v = ph.randn(g, n, Hkv, d).to(torch.bfloat16)
    turns, _ = blink.blink_rope_table(d)
    cu, start = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = blink.new_workspace(blink.paged_append_workspace_bytes(), "cuda")
    caches = [blink.blink_paged_cache(total, page, Hkv, d) for _ in range(3)]
    zeros = torch.zeros_like(v)
    took = [_median_us(lambda: blink.blink_paged_append(k, v, c, table, cu, start, n, turns=turns, interleaved=interleaved, ws=ws))
            for k, c in zip((v, zeros, -zeros), caches)]
    for c in caches[1:]:
        assert bool((c["k"].double() == 0).all())
        assert torch.equal(c["v"].view(torch.uint8), caches[0]["v"].view(torch.uint8))
    assert max(took[1:]) <= 1.5 * took[0], took
