"""Paged attention called by several host threads at once, each with its stream and workspace."""
import threading

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402


def test_calls_of_different_sizes_by_several_threads():
    """Batches of 128 and of 1024 sequences far below max_len, whose blocks take different amounts of shared memory: no
    thread's call fails for another's, and all get the same results.  The C calls themselves, so that they overlap."""
    g = ph.gen(71)
    Hq, Hkv, d, page, most, bound = 2, 1, 64, 16, 16, 131072
    row, total = ph.table_for(g, [most], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, row, [most])
    L = blink.lib()
    jobs, keep = [], []
    for S in (128, 1024, 128, 1024):
        q = ph.randn(g, S, 1, Hq, d).to(torch.bfloat16)
        table = row.expand(S, -1).contiguous()
        length = torch.randint(0, most + 1, (S,), device="cuda", generator=g).to(torch.int32)
        want, _, _ = blink.blink_paged_token_attention(q, cache, table, length, bound)
        out, stream = torch.zeros_like(q), torch.cuda.Stream()
        ws = blink.new_workspace(blink.paged_token_attention_workspace_bytes(S, 1, bound, Hq, Hkv, d), "cuda")
        jobs.append((q.data_ptr(), *(cache[n].data_ptr() for n in ("k", "v", "k_scale", "v_scale")), Hkv * page * d, Hkv, total, page,
                     table.data_ptr(), 1, 1, length.data_ptr(), S, 1, bound, Hq, Hkv, d, 0.0, out.data_ptr(), None, ws.data_ptr(),
                     ws.numel(), stream.cuda_stream))
        keep.append((want, out, table, length, q, ws, stream))
    torch.cuda.synchronize()
    failed, ready = [], threading.Barrier(len(jobs))

    def work(args):
        ready.wait()
        failed.extend(st for st in (L.blink_paged_token_attention(*args) for _ in range(3000)) if st != blink.BLINK_OK)
    threads = [threading.Thread(target=work, args=(a,)) for a in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, f"{len(failed)} of 12000 calls failed: {blink.status_string(failed[0])}"
    for want, out, *_ in keep:
        assert torch.equal(out, want)
