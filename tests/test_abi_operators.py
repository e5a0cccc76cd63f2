"""Argument checks of the key-weight, eviction and whole-vocabulary calls: each bad call is refused on the
host before anything is launched (C ABI) or before the library is reached (Python binding).  CPU only."""
import ctypes

import pytest
import torch

from shared_prefix_question_gb300 import blink, build

FAKE = 0x100000  # never dereferenced: every call below is refused on the host
INVALID, RANGE, SMALL = blink.BLINK_INVALID_ARG, blink.BLINK_OUT_OF_RANGE, blink.BLINK_WORKSPACE_TOO_SMALL
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return blink.lib()


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(lse=None), INVALID), (dict(w=None), INVALID),
    (dict(ws=None), INVALID), (dict(rows=0), INVALID), (dict(d=96), INVALID), (dict(Hq=6, Hkv=4), INVALID),
    (dict(Hq=258, Hkv=2), INVALID), (dict(P=0), RANGE), (dict(P=131073, ws_=131073), RANGE),
    (dict(stride=100), INVALID), (dict(stride=132), INVALID), (dict(lse_stride=9), INVALID),
    (dict(w_stride=63), INVALID), (dict(q=FAKE + 2), INVALID), (dict(k=FAKE + 8), INVALID),
    (dict(decay=-0.5), INVALID), (dict(decay=NAN), INVALID), (dict(decay=INF), INVALID),
    (dict(decay=0.5), INVALID),                                        # no previous weights
    (dict(decay=0.5, prev=FAKE + 0x80000 + 4), INVALID),               # overlaps the output, shifted by one
    (dict(decay=0.5, prev=FAKE + 0x80000, prev_stride=128), INVALID),  # same start, another stride
    (dict(decay=0.5, prev=FAKE, prev_stride=63), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(wsb=8), SMALL),
])
def test_key_weights_refusals(lib, bad, status):
    a = dict(q=FAKE, k=FAKE, stride=128, lse=FAKE, lse_stride=10, rows=10, P=64, Hq=4, Hkv=2, d=64, scale=0.0, decay=0.0,
             prev=None, prev_stride=64, w=FAKE + 0x80000, w_stride=64, ws=FAKE, wsb=1 << 30)
    a.update({k: v for k, v in bad.items() if k in a})
    st = lib.blink_prefix_key_weights(_p(a["q"]), _p(a["k"]), a["stride"], _p(a["lse"]), a["lse_stride"], a["rows"], a["P"],
                                      a["Hq"], a["Hkv"], a["d"], a["scale"], a["decay"], _p(a["prev"]), a["prev_stride"],
                                      _p(a["w"]), a["w_stride"], _p(a["ws"]), a["wsb"], None)
    assert st == status


K, V, KD, VD = 0x10000000, 0x20000000, 0x30000000, 0x40000000
ROW = 2 * 64 * 2  # bytes of an arena row below


@pytest.mark.parametrize("bad,status", [
    (dict(w=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kd=None), INVALID),
    (dict(vd=None), INVALID), (dict(slots=None), INVALID), (dict(ws=None), INVALID), (dict(P=0), RANGE),
    (dict(P=131073), RANGE), (dict(keep=0), RANGE), (dict(keep=101), RANGE), (dict(Hkv=0), RANGE), (dict(d=4), RANGE),
    (dict(d=1032, stride=2064, dst=2064), RANGE), (dict(d=60), INVALID), (dict(sink=-1), INVALID),
    (dict(recent=-1), INVALID), (dict(stride=120), INVALID), (dict(stride=132), INVALID), (dict(dst=120), INVALID),
    (dict(w_stride=99), INVALID), (dict(pos=FAKE, pos_stride=99), INVALID), (dict(wd=FAKE, wd_stride=39), INVALID),
    (dict(pd=FAKE, pd_stride=39), INVALID), (dict(k=K + 8), INVALID), (dict(vd=VD + 2), INVALID),
    (dict(kd=K + ROW), INVALID),             # overlaps its source by all rows but one
    (dict(kd=K, dst=256, stride=128), INVALID),  # same start, another stride
    (dict(kd=V), INVALID), (dict(vd=K), INVALID), (dict(kd=KD, vd=KD), INVALID),
    (dict(kd=KD, vd=KD + 39 * ROW), INVALID),  # the last row of one is the first of the other
    (dict(wd=0x50000000 + 4, wd_stride=100), INVALID), (dict(pos=FAKE, pd=FAKE + 8, pd_stride=100), INVALID),
    (dict(pd=0x50000000), INVALID), (dict(slots=0x50000000 + 40), INVALID), (dict(wd=FAKE, pd=FAKE + 80), INVALID),
    (dict(wsb=200), SMALL),
])
def test_evict_refusals(lib, bad, status):
    a = dict(w=0x50000000, w_stride=100, pos=None, pos_stride=100, P=100, keep=40, sink=0, recent=2**31 - 1, Hkv=2, d=64,
             k=K, v=V, stride=128, kd=KD, vd=VD, dst=128, slots=0x60000000, wd=None, wd_stride=40, pd=None, pd_stride=40,
             ws=FAKE, wsb=1 << 30)
    a.update(bad)
    st = lib.blink_kv_evict(_p(a["w"]), a["w_stride"], _p(a["pos"]), a["pos_stride"], a["P"], a["keep"], a["sink"],
                            a["recent"], a["Hkv"], a["d"], _p(a["k"]), _p(a["v"]), a["stride"], _p(a["kd"]), _p(a["vd"]),
                            a["dst"], _p(a["slots"]), _p(a["wd"]), a["wd_stride"], _p(a["pd"]), a["pd_stride"],
                            _p(a["ws"]), a["wsb"], None)
    assert st == status


@pytest.mark.parametrize("bad,status", [
    (dict(hidden=None), INVALID), (dict(W=None), INVALID), (dict(ws=None), INVALID), (dict(tg=None), INVALID),
    (dict(lp=None, en=None, lse=None, ids=None, tlp=None, top=0), INVALID), (dict(ids=None), INVALID),
    (dict(tlp=None), INVALID), (dict(top=0), INVALID), (dict(ids=None, tlp=None), INVALID), (dict(T=0.0), INVALID),
    (dict(T=-1.0), INVALID), (dict(T=NAN), INVALID), (dict(T=INF), INVALID), (dict(H=4), INVALID), (dict(H=260), INVALID),
    (dict(V=0), INVALID), (dict(rows=0), INVALID), (dict(stride=248), INVALID), (dict(stride=260), INVALID),
    (dict(hidden=FAKE + 2), INVALID), (dict(W=FAKE + 8), INVALID), (dict(top=33), RANGE), (dict(top=-1), RANGE),
    (dict(V=3), RANGE), (dict(H=32776, stride=32776), RANGE), (dict(V=(1 << 24) + 1), RANGE), (dict(n=0), RANGE),
    (dict(n=131073, rows=200000), RANGE), (dict(n=11), INVALID), (dict(wsb=256), SMALL),
])
def test_logprobs_refusals(lib, bad, status):
    a = dict(hidden=FAKE, stride=256, rows=10, idx=None, W=FAKE, V=1024, H=256, tg=FAKE, n=10, T=1.0, top=5, lp=FAKE,
             en=FAKE, lse=FAKE, ids=FAKE, tlp=FAKE, ws=FAKE, wsb=1 << 34)
    a.update(bad)
    st = lib.blink_token_logprobs(_p(a["hidden"]), a["stride"], a["rows"], _p(a["idx"]), _p(a["W"]), a["V"], a["H"],
                                  _p(a["tg"]), a["n"], a["T"], a["top"], _p(a["lp"]), _p(a["en"]), _p(a["lse"]),
                                  _p(a["ids"]), _p(a["tlp"]), _p(a["ws"]), a["wsb"], None)
    assert st == status


def test_workspace_queries(lib):
    assert blink.key_weights_workspace_bytes(10, 64, 4, 2, 64) >= 256
    assert blink.kv_evict_workspace_bytes(100, 40, 2) >= 256
    small, large = (blink.token_logprobs_workspace_bytes(n, 2560, 151936, 20) for n in (1, 4096))
    assert 256 <= small < large
    for bad in ((0, 2560, 151936, 20), (5, 2560, 0, 0), (5, 2560, 100, 33)):
        assert blink.token_logprobs_workspace_bytes(*bad) >= 256


def test_binding_refuses_host_tensors_and_shapes():
    """The binding names the argument and raises before it loads the library or touches a device."""
    bf, f32 = torch.bfloat16, torch.float32
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        blink.blink_prefix_key_weights(torch.zeros(2, 4, 64, dtype=bf), torch.zeros(8, 2, 64, dtype=bf), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="weights must be a CUDA tensor"):
        blink.blink_kv_evict(torch.zeros(2, 8), torch.zeros(8, 2, 64, dtype=bf), torch.zeros(8, 2, 64, dtype=bf), 4)
    with pytest.raises(ValueError, match="hidden must be a CUDA tensor"):
        blink.blink_token_logprobs(torch.zeros(2, 64, dtype=bf), torch.zeros(8, 64, dtype=bf))

    class Fake(torch.Tensor):  # a host tensor that says it is on a GPU: the shape and type checks come next
        is_cuda = True

    def fake(t):
        return t.as_subclass(Fake)
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        blink._need("q", fake(torch.zeros(2, 4, 64)), bf, (None, None, None))
    with pytest.raises(ValueError, match="must have shape"):
        blink._need("lse", fake(torch.zeros(4, 3)), f32, (4, 2))
    with pytest.raises(ValueError, match="contiguous"):
        blink._need("k", fake(torch.zeros(8, 64, 2, dtype=bf).transpose(1, 2)), bf, (8, 2, 64), inner=2)
    blink._need("k", fake(torch.zeros(8, 4, 64, dtype=bf)[:, :2]), bf, (8, 2, 64), inner=2)  # strided rows are fine
    with pytest.raises(ValueError, match="contiguous"):
        blink._need("weights", fake(torch.zeros(8, 2).t()), f32, (2, 8))


def test_workspaces_have_to_be_aligned(lib):
    """The scratch behind a workspace's header holds 32-bit words and rows that copies of 16 bytes read."""
    ws, n = _p(FAKE + 0x90008), 1 << 34
    a, b, c = (_p(K + i * 0x1000000) for i in range(3))
    assert lib.blink_prefix_key_weights(a, b, 128, c, 10, 10, 64, 4, 2, 64, 0.0, 0.0, None, 64, _p(FAKE + 0x80000), 64, ws, n,
                                        None) == INVALID
    assert lib.blink_kv_evict(a, 100, None, 100, 100, 40, 0, 2**31 - 1, 2, 64, _p(V), b, 128, _p(KD), _p(VD), 128, c, None, 40,
                              None, 40, ws, n, None) == INVALID
    assert lib.blink_token_logprobs(a, 256, 10, None, b, 1024, 256, None, 10, 1.0, 0, None, c, None, None, None, ws, n,
                                    None) == INVALID


def test_evict_workspace_grows_with_the_kept_keys(lib):
    sizes = [blink.kv_evict_workspace_bytes(131072, keep, 8) for keep in (1, 1000, 131072)]
    assert sizes == sorted(sizes) and sizes[-1] >= 2 * 4 * 8 * 131072
    for bad in ((100, 0, 2), (100, 10, 0), (100, -1, 2)):
        assert blink.kv_evict_workspace_bytes(*bad) >= 256


def test_binding_row_strides():
    """Of tensors without rows too (the library refuses those by their sizes)."""
    for shape in ((0, 4), (2, 0), (0, 2, 64), (3, 2, 64)):
        t = torch.zeros(shape)
        assert blink._row_stride(t) == t.stride(0)
    assert blink._row_stride(torch.zeros(1, 7).expand(1, 7)) == 7
    assert blink._row_stride(torch.zeros(4, 10)[:1, :6]) == 6


@pytest.mark.parametrize("T,status", [(1e-40, INVALID), (4.2e-39, INVALID), (4.3e-39, SMALL), (1e-30, SMALL), (3e38, SMALL)])
def test_logprobs_temperature_without_a_reciprocal(lib, T, status):
    """log2(e) / temperature has to be a number; what passes that check is refused for its workspace here."""
    st = lib.blink_token_logprobs(_p(FAKE), 256, 10, None, _p(FAKE), 1024, 256, _p(FAKE), 10, T, 0, _p(FAKE), None, None, None,
                                  None, _p(FAKE), 256, None)
    assert st == status


def test_binding_refuses_what_32_bits_do_not_hold():
    """ctypes drops the bits above 32 of a number: 2^32 + 5 would be passed as 5."""
    class Fake(torch.Tensor):  # a host tensor that says it is on a GPU: the checks of the arguments come first
        is_cuda = True

    def fake(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype).as_subclass(Fake)
    w, k, v = fake(2, 8, dtype=torch.float32), fake(8, 2, 64), fake(8, 2, 64)
    for kw in (dict(sink=2**32), dict(recent_from=2**32 + 5), dict(recent_from=2**31), dict(sink=-2**31 - 1)):
        with pytest.raises(ValueError, match="must fit 32 bits"):
            blink.blink_kv_evict(w, k, v, 4, **kw)
    with pytest.raises(TypeError):
        blink.blink_kv_evict(w, k, v, 4, sink=1.5)
    h, u = fake(2, 8), fake(9, 8)
    with pytest.raises(ValueError, match="must fit 32 bits"):
        blink.blink_token_logprobs(h, u, top=2**32 + 1)
    long = fake(8).as_strided((2**32 + 4, 8), (0, 1))
    with pytest.raises(ValueError, match="must fit 32 bits"):
        blink.blink_token_logprobs(long, u)
