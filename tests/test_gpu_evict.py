"""Eviction against a numpy selection: slots, positions and copies are exact."""
import numpy as np
import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def want_slots(w, pos, keep, sink, recent_from):
    Hkv, P = w.shape
    out = np.empty((Hkv, keep), np.int32)
    for h in range(Hkv):
        wh = np.where(np.isnan(w[h]), -np.inf, w[h].astype(np.float64))
        nan_last = np.isnan(w[h])
        guarded = (pos[h] < sink) | (pos[h] >= recent_from)
        kept = np.sort(np.lexsort((np.arange(P), nan_last, -wh, ~guarded))[:keep])
        out[h] = np.arange(keep)
        holes = np.setdiff1d(np.arange(keep), kept[kept < keep])
        out[h, holes] = kept[kept >= keep]
    return out


def inputs(P, Hkv, d, seed, kind="normal"):
    rng = np.random.default_rng(seed)
    w = rng.lognormal(0, 2, (Hkv, P)).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 4, (Hkv, P)).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "zeros":
        w[rng.random((Hkv, P)) < 0.9] = 0.0
        w[rng.random((Hkv, P)) < 0.3] *= -1.0  # among them -0, equal to 0, and negative weights
    elif kind == "special":
        w[rng.random((Hkv, P)) < 0.1] = np.nan
        w[rng.random((Hkv, P)) < 0.05] = np.inf
        w[rng.random((Hkv, P)) < 0.05] = -np.inf
        w[rng.random((Hkv, P)) < 0.05] = 1e-42  # subnormal
    elif kind == "ascending":
        w[:] = np.arange(P, dtype=np.float32)
    elif kind == "descending":
        w[:] = -np.arange(P, dtype=np.float32)
    k = torch.from_numpy(rng.integers(-2**15, 2**15, (P, Hkv, d)).astype(np.int16)).cuda()
    v = torch.from_numpy(rng.integers(-2**15, 2**15, (P, Hkv, d)).astype(np.int16)).cuda()
    return w, k.view(BF), v.view(BF)  # every bit pattern, NaN among them: copies are compared as bits


def bits(t):
    return t.contiguous().view(torch.int16)


def run_and_check(w, k, v, keep, pos=None, sink=0, recent_from=None, in_place=False):
    Hkv, P = w.shape
    d = k.shape[2]
    p_np = np.tile(np.arange(P, dtype=np.int32), (Hkv, 1)) if pos is None else pos
    slots = want_slots(w, p_np, keep, sink, 2**31 - 1 if recent_from is None else recent_from)
    st = torch.from_numpy(slots).cuda().long()
    head = torch.arange(Hkv, device="cuda")
    wk, wv = bits(k)[st.t(), head].clone(), bits(v)[st.t(), head].clone()
    wt = torch.from_numpy(w).cuda()
    pt = None if pos is None else torch.from_numpy(pos).cuda()
    k0, v0 = bits(k).clone(), bits(v).clone()
    if in_place:
        r = blink.blink_kv_evict(wt, k, v, keep, pos=pt, sink=sink, recent_from=recent_from, weights_dst=wt[:, :keep],
                                 pos_dst=None if pt is None else pt[:, :keep])
        assert r["k"].data_ptr() == k.data_ptr()
        assert torch.equal(bits(k)[keep:], k0[keep:]) and torch.equal(bits(v)[keep:], v0[keep:])  # left as they were
    else:
        kd = torch.zeros(keep, Hkv, d, dtype=BF, device="cuda")
        vd = torch.zeros_like(kd)
        r = blink.blink_kv_evict(wt, k, v, keep, pos=pt, sink=sink, recent_from=recent_from, k_dst=kd, v_dst=vd)
        assert torch.equal(bits(k), k0) and torch.equal(bits(v), v0)
    assert np.array_equal(r["slots"].cpu().numpy(), slots)
    assert torch.equal(bits(r["k"]), wk) and torch.equal(bits(r["v"]), wv)
    hn = np.arange(Hkv)[:, None]
    assert np.array_equal(r["weights"].cpu().numpy(), w[hn, slots], equal_nan=True)
    assert np.array_equal(r["pos"].cpu().numpy(), p_np[hn, slots])
    return r


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("P,keep,Hkv,d", [(1, 1, 1, 64), (2, 1, 1, 8), (64, 32, 2, 64), (64, 64, 2, 64), (65, 1, 3, 128),
                                          (1000, 999, 2, 64), (1024, 500, 1, 128), (1025, 512, 5, 64),
                                          (2049, 2000, 8, 128), (8191, 77, 4, 64), (8193, 4000, 2, 72)])
def test_sizes(P, keep, Hkv, d, in_place):
    w, k, v = inputs(P, Hkv, d, seed=P + keep)
    run_and_check(w, k, v, keep, in_place=in_place)


@pytest.mark.parametrize("kind", ["ties", "equal", "zeros", "special", "ascending", "descending"])
@pytest.mark.parametrize("P,keep", [(300, 120), (5000, 1234), (20000, 19000)])
def test_ties_and_special_weights(kind, P, keep):
    w, k, v = inputs(P, 2, 64, seed=5, kind=kind)
    run_and_check(w, k, v, keep, in_place=True)


@pytest.mark.parametrize("keep", [700, 3000, 131071])
def test_longest_prefix(keep):
    w, k, v = inputs(131072, 2, 64, seed=keep, kind="zeros")
    run_and_check(w, k, v, keep, in_place=True)


@pytest.mark.parametrize("sink,recent,keep", [(4, 64, 500), (0, 900, 500), (600, 0, 500), (0, 500, 500), (1, 1, 2)])
def test_protected_positions(sink, recent, keep):
    """Fewer protected keys than `keep`, exactly as many, and more of them."""
    w, k, v = inputs(3000, 2, 64, seed=sink + recent, kind="special")
    run_and_check(w, k, v, keep, sink=sink, recent_from=3000 - recent)


def test_repeated_eviction_carries_positions():
    """Evict twice: the second call sees the first's positions, out of slot order, and protects by them."""
    w, k, v = inputs(4000, 3, 64, seed=1)
    k0, v0 = bits(k).clone(), bits(v).clone()
    wt = torch.from_numpy(w).cuda()
    pt = torch.arange(4000, dtype=torch.int32, device="cuda").repeat(3, 1)
    blink.blink_kv_evict(wt, k, v, 1500, pos=pt, sink=4, recent_from=3900, weights_dst=wt[:, :1500], pos_dst=pt[:, :1500])
    w2, p2 = wt[:, :1500].cpu().numpy(), pt[:, :1500].cpu().numpy()
    assert all(set(range(4)) | set(range(3900, 4000)) <= set(p2[h]) for h in range(3))
    r = run_and_check(w2, k[:1500], v[:1500], 333, pos=p2, sink=4, recent_from=3900, in_place=True)
    pos = r["pos"].long()
    head = torch.arange(3, device="cuda")
    assert torch.equal(bits(k[:333]), k0[pos.t(), head])  # each key is still the one of its position
    assert torch.equal(bits(v[:333]), v0[pos.t(), head])


def test_strided_and_interleaved_arena():
    """K and V interleaved in one arena row, and wider rows: in place and into another region of it."""
    w, k, v = inputs(900, 2, 64, seed=2)
    arena = torch.zeros(2000, 5, 64, dtype=BF, device="cuda")  # heads 0-1: K, 2-3: V, 4: something else
    arena[:900, 0:2] = k
    arena[:900, 2:4] = v
    arena[:, 4] = 7.0
    ka, va = arena[:900, 0:2], arena[:900, 2:4]
    run_and_check(w, ka, va, 400, in_place=True)
    arena[:900, 0:2] = k
    arena[:900, 2:4] = v
    wt = torch.from_numpy(w).cuda()
    r = blink.blink_kv_evict(wt, ka, va, 400, k_dst=arena[1000:1400, 0:2], v_dst=arena[1000:1400, 2:4])
    assert torch.equal(bits(ka), bits(k)) and torch.equal(bits(va), bits(v))
    st, head = r["slots"].long(), torch.arange(2, device="cuda")
    assert torch.equal(bits(arena[1000:1400, 0:2]), bits(k)[st.t(), head])
    assert torch.equal(bits(arena[1000:1400, 2:4]), bits(v)[st.t(), head])
    assert bool((arena[:, 4] == 7.0).all()) and bool((arena[1400:, :4] == 0).all())


def test_overlapping_destination_is_refused():
    w, k, v = inputs(100, 2, 64, seed=3)
    wt = torch.from_numpy(w).cuda()
    with pytest.raises(blink.BlinkError) as e:
        blink.blink_kv_evict(wt, k, v, 40, k_dst=k[1:41], v_dst=torch.zeros_like(v[:40]))
    assert e.value.status == blink.BLINK_INVALID_ARG


def test_repeat_bitwise_own_stream_and_graph():
    w, k, v = inputs(30000, 4, 128, seed=4, kind="ties")
    wt = torch.from_numpy(w).cuda()
    kd, vd = torch.zeros_like(k[:7000]), torch.zeros_like(v[:7000])
    r = blink.blink_kv_evict(wt, k, v, 7000, k_dst=kd, v_dst=vd)
    want = r["slots"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r2 = blink.blink_kv_evict(wt, k, v, 7000, k_dst=kd, v_dst=vd, stream=side)
    side.synchronize()
    assert torch.equal(r2["slots"], want)
    ws = blink.new_workspace(blink.kv_evict_workspace_bytes(30000, 7000, 4), "cuda")
    slots = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blink.blink_kv_evict(wt, k, v, 7000, k_dst=kd, v_dst=vd, slots=slots, ws=ws)
    wt.copy_(torch.from_numpy(inputs(30000, 4, 128, seed=14, kind="zeros")[0]).cuda())
    graph.replay()
    torch.cuda.synchronize()
    pos = np.tile(np.arange(30000, dtype=np.int32), (4, 1))
    assert np.array_equal(slots.cpu().numpy(), want_slots(wt.cpu().numpy(), pos, 7000, 0, 2**31 - 1))
    assert torch.equal(bits(kd), bits(k)[slots.long().t(), torch.arange(4, device="cuda")])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("P,keep,Hkv,d", [(40, 17, 64, 8), (300, 100, 65, 8), (300, 299, 130, 16), (4096, 2048, 2, 64),
                                          (4097, 2049, 3, 64), (16385, 8000, 2, 64), (16896, 16000, 5, 64),
                                          (32769, 5, 2, 64), (32768, 32767, 1, 64)])
def test_many_heads_and_piece_edges(P, keep, Hkv, d, in_place):
    """More heads than a moving block takes, and lengths at the edges of the blocks' pieces."""
    w, k, v = inputs(P, Hkv, d, seed=P + Hkv, kind="zeros")
    run_and_check(w, k, v, keep, in_place=in_place)


def test_a_workspace_carries_nothing_over():
    """Calls of other sizes with one workspace, its scratch full of other values: as with a new one."""
    ws = torch.full((blink.kv_evict_workspace_bytes(9000, 4500, 4),), 0x5A, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    for P, keep, Hkv in ((9000, 4500, 4), (700, 33, 2), (9000, 100, 4), (5000, 4500, 1)):
        w, k, v = inputs(P, Hkv, 64, seed=P + keep)
        wt = torch.from_numpy(w).cuda()
        kd, vd = (torch.zeros(keep, Hkv, 64, dtype=BF, device="cuda") for _ in range(2))
        r = blink.blink_kv_evict(wt, k, v, keep, k_dst=kd, v_dst=vd, ws=ws)
        assert np.array_equal(r["slots"].cpu().numpy(),
                              want_slots(w, np.tile(np.arange(P, dtype=np.int32), (Hkv, 1)), keep, 0, 2**31 - 1))
    assert blink.blink_read_device_status(ws) == blink.BLINK_OK


def test_no_recent_position_is_protected_by_default():
    """Not even the largest there is, when the first positions are."""
    w, k, v = inputs(500, 2, 64, seed=9)
    pos = np.tile(np.arange(500, dtype=np.int32), (2, 1))
    pos[:, 100:200] = 2**31 - 1
    want = want_slots(w, pos.astype(np.int64), 60, 5, 2**31)
    r = blink.blink_kv_evict(torch.from_numpy(w).cuda(), k, v, 60, pos=torch.from_numpy(pos).cuda(), sink=5)
    assert np.array_equal(r["slots"].cpu().numpy(), want)


def test_one_key_kept_in_its_strided_region():
    """A destination that is row 0 of the source is in place whatever the rows' stride."""
    w, k, v = inputs(70, 2, 64, seed=10)
    arena = torch.zeros(70, 4, 64, dtype=BF, device="cuda")
    arena[:, :2], arena[:, 2:] = k, v
    r = blink.blink_kv_evict(torch.from_numpy(w).cuda(), arena[:, :2], arena[:, 2:], 1, k_dst=arena[:1, :2],
                             v_dst=arena[:1, 2:])
    best = torch.from_numpy(w.argmax(1)).cuda()
    head = torch.arange(2, device="cuda")
    assert torch.equal(r["slots"][:, 0].long(), best)
    assert torch.equal(bits(arena[0, :2]), bits(k)[best, head]) and torch.equal(bits(arena[0, 2:]), bits(v)[best, head])
    assert torch.equal(bits(arena[1:, :2]), bits(k)[1:]) and torch.equal(bits(arena[1:, 2:]), bits(v)[1:])


def test_two_graphs_of_one_workspace_and_two_streams():
    """Replays in turn share a workspace; calls at the same time have one each."""
    cases = []
    for P, keep, seed in ((6000, 2500, 21), (20000, 900, 22)):
        w, k, v = inputs(P, 3, 64, seed=seed)
        kd, vd = (torch.zeros(keep, 3, 64, dtype=BF, device="cuda") for _ in range(2))
        slots = torch.empty(3, keep, dtype=torch.int32, device="cuda")
        want = want_slots(w, np.tile(np.arange(P, dtype=np.int32), (3, 1)), keep, 0, 2**31 - 1)
        cases.append((torch.from_numpy(w).cuda(), k, v, keep, kd, vd, slots, want))
    ws = blink.new_workspace(max(blink.kv_evict_workspace_bytes(w.shape[1], keep, 3) for w, _, _, keep, *_ in cases), "cuda")
    graphs = []
    for w, k, v, keep, kd, vd, slots, _ in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            blink.blink_kv_evict(w, k, v, keep, k_dst=kd, v_dst=vd, slots=slots, ws=ws)
        graphs.append(graph)
    for _ in range(3):
        for graph, (*_, slots, want) in zip(graphs, cases):
            slots.fill_(-1)
            graph.replay()
            assert np.array_equal(slots.cpu().numpy(), want)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (w, k, v, keep, kd, vd, slots, _) in zip(streams, cases):
            blink.blink_kv_evict(w, k, v, keep, k_dst=kd, v_dst=vd, slots=slots, stream=s)
    torch.cuda.synchronize()
    head = torch.arange(3, device="cuda")
    for w, k, v, keep, kd, vd, slots, want in cases:
        assert np.array_equal(slots.cpu().numpy(), want)
        st = slots.long().t()
        assert torch.equal(bits(kd), bits(k)[st, head]) and torch.equal(bits(vd), bits(v)[st, head])
