"""Evictions one behind the other over one workspace, with nothing between them on the stream: each call's
move is resident while its own selection rewrites the lists that the call before has left."""
import numpy as np
import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu


def want_slots(w, keep):
    out = np.empty((w.shape[0], keep), np.int32)
    for h in range(w.shape[0]):
        kept = np.sort(np.lexsort((np.arange(w.shape[1]), -w[h]))[:keep])
        out[h] = np.arange(keep)
        out[h, np.setdiff1d(np.arange(keep), kept[kept < keep])] = kept[kept >= keep]
    return out


@pytest.mark.parametrize("P,keep,Hkv", [(700, 300, 2), (18432, 9216, 8), (5000, 4999, 3), (2000, 1, 5)])
@pytest.mark.parametrize("captured", [False, True])
def test_calls_in_a_row(P, keep, Hkv, captured):
    rng = np.random.default_rng(P)
    ws_np = [rng.lognormal(0, 2, (Hkv, P)).astype(np.float32) for _ in range(4)]
    ws_np.append(np.tile(np.arange(P, dtype=np.float32), (Hkv, 1)))  # every kept key moves, as far as they can
    ws_np.append(-ws_np[-1])                                         # none moves
    weights = [torch.from_numpy(w).cuda() for w in ws_np]
    k = torch.randn(P, Hkv, 64, device="cuda").to(torch.bfloat16)
    v = torch.randn(P, Hkv, 64, device="cuda").to(torch.bfloat16)
    slots = [torch.empty(Hkv, keep, dtype=torch.int32, device="cuda") for _ in weights]
    dst = [(torch.empty(keep, Hkv, 64, dtype=torch.bfloat16, device="cuda"),
            torch.empty(keep, Hkv, 64, dtype=torch.bfloat16, device="cuda")) for _ in weights]
    ws = blink.new_workspace(blink.kv_evict_workspace_bytes(P, keep, Hkv), "cuda")

    def calls():
        for w, s, (kd, vd) in zip(weights, slots, dst):
            blink.blink_kv_evict(w, k, v, keep, k_dst=kd, v_dst=vd, slots=s, ws=ws)
    calls()
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        for s in slots:
            s.fill_(-1)
        for _ in range(3):
            graph.replay()
    head = torch.arange(Hkv, device="cuda")
    for w, s, (kd, vd) in zip(ws_np, slots, dst):
        want = torch.from_numpy(want_slots(w, keep)).cuda()
        assert torch.equal(s, want)
        at = want.long().t()
        assert torch.equal(kd, k[at, head]) and torch.equal(vd, v[at, head])
