"""Calls of the three operators that are rare but allowed: the first call of a process inside a graph capture, a
last launch of one row, very many rows against few keys."""
import math
import os
import subprocess
import sys

import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST_CALL = """
import torch
from shared_prefix_question_gb300 import blink
torch.manual_seed(0)
what = {what!r}
bf = torch.bfloat16
a = torch.randn(300, 8, 128, device="cuda").to(bf)
k, v = torch.randn(700, 2, 128, device="cuda").to(bf), torch.randn(700, 2, 128, device="cuda").to(bf)
lse = torch.full((8, 300), 8.0, device="cuda")
w = torch.rand(2, 700, device="cuda")
kd, vd = torch.empty(100, 2, 128, dtype=bf, device="cuda"), torch.empty(100, 2, 128, dtype=bf, device="cuda")
h, u = torch.randn(200, 256, device="cuda").to(bf), torch.randn(999, 256, device="cuda").to(bf)
blink.lib()
ws = blink.new_workspace(16 << 20, "cuda")
def call():
    if what == "weights":
        return [blink.blink_prefix_key_weights(a, k, lse, ws=ws)[0]]
    if what == "evict":
        r = blink.blink_kv_evict(w, k, v, 100, k_dst=kd, v_dst=vd, ws=ws)
        return [r["slots"], r["k"], r["weights"]]
    r = blink.blink_token_logprobs(h, u, top=5, ws=ws)
    return [r["entropy"], r["lse"], r["top_ids"], r["top_logprobs"]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out]
assert all(torch.equal(x, y) for x, y in zip(got, call()))
print("same")
"""


@pytest.mark.parametrize("what", ["weights", "evict", "logprobs"])
def test_the_first_call_of_a_process_is_captured(what):
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(what=what)], cwd=ROOT, capture_output=True, text=True,
                       timeout=240)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("n", [8193, 8192 + 129, 2 * 8192 + 1])
def test_a_last_launch_of_few_rows(n):
    """Exact logits; the last launch is of another form than the ones before it."""
    g = torch.Generator(device="cuda").manual_seed(n)
    h = (torch.randint(-8, 9, (n, 64), device="cuda", generator=g) / 8.0).to(BF)
    W = (torch.randint(-16, 17, (1025, 64), device="cuda", generator=g) / 64.0).to(BF)
    idx = torch.randperm(n, device="cuda", generator=g).to(torch.int32)
    ids = torch.sort(h.double() @ W.double().t(), dim=1, descending=True, stable=True)[1][:, :7].to(torch.int32)
    ws = blink.new_workspace(blink.token_logprobs_workspace_bytes(n, 64, 1025, 7), "cuda")
    guard = ws.numel()
    room = torch.full((guard + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    room[:256] = 0
    r = blink.blink_token_logprobs(h, W, row_idx=idx, top=7, ws=room[:guard])
    assert torch.equal(r["top_ids"], ids[idx.long()])
    assert bool((room[guard:] == 0x5A).all())
    direct = blink.blink_token_logprobs(h, W, top=7, ws=room[:guard])
    assert torch.equal(direct["top_ids"], ids)


@pytest.mark.parametrize("rows,Hq,Hkv,d,P", [(100001, 1, 1, 64, 40), (60000, 4, 2, 128, 300), (40000, 5, 1, 64, 1)])
def test_many_rows_against_few_keys(rows, Hq, Hkv, d, P):
    """One or two units of keys, cut over all blocks.  Bound: each block adds its tiles in a row, the join the blocks;
    the exponent is off by d / 16 steps of 2^-22 of sums below max |s| and a few roundings of |s| and |lse|."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    q = torch.randn(rows, Hq, d, device="cuda", generator=g).to(BF)
    k = torch.randn(P, Hkv, d, device="cuda", generator=g).to(BF)
    grp = Hq // Hkv
    s = torch.einsum("thgd,phd->hgtp", q.double().view(rows, Hkv, grp, d), k.double()) / math.sqrt(d)
    lse = torch.logsumexp(s, -1).view(Hq, rows).float()
    w, ws = blink.blink_prefix_key_weights(q, k, lse)
    want = (s - lse.double().view(Hkv, grp, rows, 1)).exp().sum((1, 2))
    tiles = -(-rows // (128 // grp))
    mag = float(s.abs().max()) * 4 + float(lse.abs().max())  # partial sums of a product within four times it
    tol = 2.0**-22 * (d / 16 * mag + 1) + 2.0**-24 * (6 * mag + tiles + 16 + 152)
    assert float(((w.double() - want) / want).abs().max()) <= tol
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK
