"""The cache-eviction path as a serving program runs it: attention over an arena prefix, the weight each key
received, eviction in place, attention over what is left, and the whole-vocabulary readout that says what the
eviction cost.  Each step is compared with its formula in 64 bits on the same inputs."""
import math

import numpy as np
import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def dense(q, k, v, kt, vt, cu, allowed):
    """Attention of every tail row over the allowed prefix keys [Hkv, P] and its own tail, in 64 bits:
    out [rows, Hq, d], lse [Hq, rows], prefix weights [Hkv, P]."""
    rows, Hq, d = q.shape
    Hkv, P = allowed.shape
    g = Hq // Hkv
    out = torch.zeros(rows, Hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((Hq, rows), -math.inf, dtype=torch.float64, device=q.device)
    w = torch.zeros(Hkv, P, dtype=torch.float64, device=q.device)
    for b in range(len(cu) - 1):
        lo, hi = cu[b], cu[b + 1]
        n = hi - lo
        causal = torch.tril(torch.ones(n, n, dtype=torch.bool, device=q.device))
        for h in range(Hq):
            kv = h // g
            s = q[lo:hi, h].double() @ torch.cat([k[:, kv], kt[lo:hi, kv]]).double().t() / math.sqrt(d)
            s[:, :P].masked_fill_(~allowed[kv], -math.inf)
            s[:, P:].masked_fill_(~causal, -math.inf)
            lse[h, lo:hi] = torch.logsumexp(s, 1)
            p = (s - lse[h, lo:hi, None]).exp()
            out[lo:hi, h] = p @ torch.cat([v[:, kv], vt[lo:hi, kv]]).double()
            w[kv] += p[:, :P].sum(0)
    return out, lse, w


@pytest.mark.parametrize("P,keep,Hq,Hkv,d,lens", [(700, 300, 8, 2, 128, [5, 1, 40, 17]), (130, 64, 5, 1, 64, [3, 33]),
                                                  (1000, 999, 4, 4, 64, [20])])
def test_attention_weights_eviction_attention_readout(P, keep, Hq, Hkv, d, lens):
    g = torch.Generator(device="cuda").manual_seed(P)
    rows = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=g).to(BF)
    q, kt, vt = rand(rows, Hq, d), rand(rows, Hkv, d), rand(rows, Hkv, d)
    arena_k, arena_v = rand(P + 50, Hkv, d), rand(P + 50, Hkv, d)  # the request's region: slots 20 .. 20 + P
    k, v = arena_k[20:20 + P], arena_v[20:20 + P]
    k0, v0 = k.clone(), v.clone()
    outside = arena_k[:20].clone(), arena_k[20 + P:].clone(), arena_v[20 + P:].clone()
    cu_dev = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def attend(n):
        out, lse, ws = blink.blink_prefix_tail_attention(q, arena_k[20:20 + n], arena_v[20:20 + n], kt, vt, cu_dev,
                                                         B=len(lens), P=n, max_tail=max(lens), want_lse=True)
        assert blink.blink_read_device_status(ws) == blink.BLINK_OK
        return out, lse

    everything = torch.ones(Hkv, P, dtype=torch.bool, device="cuda")
    out, lse = attend(P)
    ref_out, ref_lse, ref_w = dense(q, k0, v0, kt, vt, cu, everything)
    w, _ = blink.blink_prefix_key_weights(q, k, lse)
    # lse is off by at most 2e-3 relative here (the attention's own tolerance), and every term with it
    assert float(((w.double() - ref_w).abs() / ref_w).max()) <= 2e-3 * max(1.0, float(ref_lse.abs().max()))

    r = blink.blink_kv_evict(w, k, v, keep, sink=2, recent_from=P - 3, weights_dst=w[:, :keep])
    kept = torch.zeros_like(everything).scatter_(1, r["pos"].long(), True)
    assert bool((kept.sum(1) == keep).all()) and bool(kept[:, :2].all()) and bool(kept[:, P - 3:].all())
    head = torch.arange(Hkv, device="cuda")
    assert torch.equal(k[:keep].view(torch.int16), k0[r["pos"].long().t(), head].view(torch.int16))
    for now, then in zip((arena_k[:20], arena_k[20 + P:], arena_v[20 + P:]), outside):
        assert torch.equal(now, then)  # the neighbours' regions

    small_out, small_lse = attend(keep)
    want_out, want_lse, want_w = dense(q, k0, v0, kt, vt, cu, kept)
    assert float((small_out.double() - want_out).abs().max()) <= 2e-2 * float(want_out.abs().max())
    assert float((small_lse.double() - want_lse).abs().max()) <= 2e-3 * max(1.0, float(want_lse.abs().max()))
    assert torch.all(small_lse.double() <= lse.double() + 1e-3)  # fewer keys, less mass

    # the second pass's weights come on top of what the kept keys gathered before
    w2, _ = blink.blink_prefix_key_weights(q, k[:keep], small_lse, prev=w[:, :keep], decay=0.5)
    want2 = 0.5 * r["weights"].double() + torch.gather(want_w, 1, r["pos"].long())
    assert float(((w2.double() - want2).abs() / want2).max()) <= 2e-3 * max(1.0, float(want_lse.abs().max()))

    # answer positions through the whole vocabulary, before and after
    V, H = 501, Hq * d
    W = (rand(V, H).float() / math.sqrt(H)).to(BF)
    last = torch.tensor([c - 1 for c in cu[1:]], dtype=torch.int32, device="cuda")
    for o in (out, small_out):
        t = torch.randint(0, V, (len(lens),), device="cuda", generator=g, dtype=torch.int32)
        res = blink.blink_token_logprobs(o.view(rows, H), W, targets=t, row_idx=last, top=3)
        z = o.view(rows, H)[last.long()].double() @ W.double().t()
        ref = torch.log_softmax(z, 1)
        assert torch.allclose(res["logprob"].double(), torch.gather(ref, 1, t.long()[:, None]).squeeze(1), atol=1e-4)
        assert torch.allclose(res["entropy"].double(), -(ref.exp() * ref).sum(1), atol=1e-4)
        assert torch.allclose(res["top_logprobs"].double(), torch.topk(ref, 3).values, atol=1e-4)


def test_weights_of_one_request_of_a_padded_batch():
    """Rows of a right-padded batch that no question owns have lse -inf from the attention; their q is garbage.
    The first request's rows are a slice of the launch."""
    Hq, Hkv, d, P = 4, 2, 64, 150
    g = torch.Generator(device="cuda").manual_seed(3)
    starts, lens = [0, 16, 32], [9, 16, 4]
    rows = 48
    q = torch.randn(rows, Hq, d, device="cuda", generator=g).to(BF)
    kt, vt = (torch.randn(rows, Hkv, d, device="cuda", generator=g).to(BF) for _ in range(2))
    k, v = (torch.randn(P, Hkv, d, device="cuda", generator=g).to(BF) for _ in range(2))
    owned = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for s, n in zip(starts, lens):
        owned[s:s + n] = True
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    ss = torch.tensor(starts, dtype=torch.int32, device="cuda")
    _, lse, ws = blink.blink_prefix_tail_attention(q, k, v, kt, vt, cu, B=3, P=P, max_tail=16, seq_start=ss, want_lse=True)
    assert bool(torch.isneginf(lse[:, ~owned]).all())
    q[~owned] = float("nan")
    for lo, hi in ((0, rows), (0, 32), (16, 48), (40, 48)):  # the last has no owned row at all
        w, _ = blink.blink_prefix_key_weights(q[lo:hi], k, lse[:, lo:hi])
        m = owned[lo:hi]
        s = torch.einsum("thgd,phd->hgtp", q[lo:hi][m].double().view(-1, Hkv, Hq // Hkv, d), k.double()) / math.sqrt(d)
        want = (s - lse[:, lo:hi][:, m].double().view(Hkv, Hq // Hkv, -1, 1)).exp().sum((1, 2))
        assert torch.allclose(w.double(), want, rtol=1e-5, atol=0)


def test_offsets_beyond_32_bits():
    """An arena whose last rows lie more than 2^31 elements from its first."""
    P, Hkv, d, stride = 70000, 1, 64, 32768
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 10 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(9)
    ka, va = (torch.zeros(P, stride, dtype=BF, device="cuda") for _ in range(2))
    k0, v0 = (torch.randn(P, Hkv * d, device="cuda", generator=g).to(BF) for _ in range(2))
    ka[:, 64:128], va[:, 64:128] = k0, v0
    k, v = ka[:, 64:128].unflatten(1, (Hkv, d)), va[:, 64:128].unflatten(1, (Hkv, d))
    q = torch.randn(2, 2, d, device="cuda", generator=g).to(BF)
    s = torch.einsum("thd,pd->htp", q.double(), k0.double()) / math.sqrt(d)
    lse = torch.logsumexp(s, -1).float()
    w, _ = blink.blink_prefix_key_weights(q, k, lse)
    want = (s - lse.double()[:, :, None]).exp().sum((0, 1))
    assert torch.allclose(w[0].double(), want, rtol=1e-4, atol=0)
    keep = 1000
    order = torch.sort(w[0].double(), descending=True, stable=True).indices[:keep]
    r = blink.blink_kv_evict(w, k, v, keep)
    assert set(r["pos"][0].tolist()) == set(order.tolist())
    pos = r["pos"][0].long()
    assert torch.equal(k[:keep, 0].view(torch.int16), k0[pos].view(torch.int16))
    assert torch.equal(v[:keep, 0].view(torch.int16), v0[pos].view(torch.int16))
    assert bool((ka[:, :64] == 0).all()) and bool((ka[:, 128:] == 0).all())
