"""Calls whose tensor maps the host encodes, made by a thread that has called nothing of CUDA before."""
import threading

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402


@pytest.mark.parametrize("kind", ["token", "few tails", "tails", "prefix tail", "many requests", "key weights", "log probabilities"])
def test_first_call_of_a_thread(kind):
    """The same bits as on the main thread.  Inputs, workspaces and the blocks of the outputs are there before, so that nothing
    but the call gives the thread its context."""
    g = ph.gen(74)
    Hq, Hkv, d, page, P = 4, 2, 64, 16, 200
    rows = 3 if kind == "few tails" else 100
    table, total = ph.table_for(g, [P], page)
    cache = ph.new_cache(g, total, Hkv, page, d)
    ph.fill(g, cache, table, [P])
    q, kt, vt = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    kp, vp = (ph.randn(g, P, Hkv, d).to(torch.bfloat16) for _ in range(2))
    cu, length = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, rows], [P]))
    hidden, unembed = ph.randn(g, rows, 256).to(torch.bfloat16), ph.randn(g, 1000, 256).to(torch.bfloat16)
    lse = blink.blink_prefix_tail_attention(q, kp, vp, kt, vt, cu, 1, P, rows, want_lse=True)[1]
    ws = blink.new_workspace(1 << 22, "cuda")
    calls = {
        "token": lambda: blink.blink_paged_token_attention(q[:1].view(1, 1, Hq, d), cache, table, length, P, want_lse=True, ws=ws)[:2],
        "tails": lambda: blink.blink_paged_prefix_tail_attention(q, cache, table, [P], kt, vt, cu, 1, rows, want_lse=True, ws=ws)[:2],
        "prefix tail": lambda: blink.blink_prefix_tail_attention(q, kp, vp, kt, vt, cu, 1, P, rows, want_lse=True, ws=ws)[:2],
        "many requests": lambda: blink.blink_prefix_tail_attention_multi(q, kp, vp, kt, vt, cu, 1, [0, rows, rows], [0, 50], [P, 20],
                                                                         rows, want_lse=True, ws=ws)[:2],
        "key weights": lambda: blink.blink_prefix_key_weights(q, kp, lse, ws=ws)[:1],
        "log probabilities": lambda: [blink.blink_token_logprobs(hidden, unembed, top=3, ws=ws)[n] for n in ("entropy", "lse", "top_ids")],
    }
    call = calls["tails" if kind == "few tails" else kind]
    for _ in range(2):  # the allocator's blocks for the thread's outputs
        want = [x.clone() for x in call()]
    torch.cuda.synchronize()
    got, stream = [], torch.cuda.current_stream()

    def work():
        try:
            got.append(call())
        except Exception as e:  # raised by the main thread
            got.append(e)
    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    if isinstance(got[0], Exception):
        raise got[0]
    stream.synchronize()
    for a, b in zip(got[0], want):
        assert torch.equal(a, b)
