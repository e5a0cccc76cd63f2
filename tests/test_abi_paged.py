"""Argument checks of the rotary and paged-cache calls (each bad call is refused on the host before anything is
launched), the table of frequencies, and workspaces.  CPU only."""
import ctypes
import math

import pytest
import torch

from shared_prefix_question_gb300 import blink, build

FAKE = 0x100000  # never dereferenced: every call below is refused on the host
INVALID, RANGE, SMALL, OK = blink.BLINK_INVALID_ARG, blink.BLINK_OUT_OF_RANGE, blink.BLINK_WORKSPACE_TOO_SMALL, blink.BLINK_OK
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return blink.lib()


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


@pytest.mark.parametrize("scaling,args,formula", [
    (None, {}, lambda t, n: t),
    ("linear", dict(factor=4.0), lambda t, n: t / 4),
    ("by_turns", dict(factor=8.0, original=8192, low=1.0, high=4.0),
     lambda t, n: (lambda s: s * t + (1 - s) * t / 8)(min(1.0, max(0.0, (8192 * t / (2 * math.pi) - 1) / 3)))),
])
@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (512, 1e6)])
def test_table(lib, scaling, args, formula, rot, base):
    turns, amplitude = blink.blink_rope_table(rot, base, scaling=scaling, device="cpu", **args)
    assert turns.dtype == torch.int64 and turns.shape == (rot // 2,) and amplitude == 1.0
    for i in range(rot // 2):
        theta = formula(base ** (-2 * i / rot), i)
        assert abs(int(turns[i]) / 2**64 * 2 * math.pi / theta - 1) <= 1e-14 + 2.0 ** -64 / theta * 8


def test_table_by_dim_and_base(lib):
    turns, amplitude = blink.blink_rope_table(128, 10000.0, scaling="by_dim", factor=16.0, original=4096, device="cpu")
    assert abs(amplitude - (0.1 * math.log(16) + 1)) < 1e-6
    plain, _ = blink.blink_rope_table(128, 10000.0, device="cpu")
    ratio = (plain.double() / turns.double()).tolist()
    assert ratio[0] == 1.0 and abs(ratio[-1] - 16) < 1e-9 and all(a <= b + 1e-9 for a, b in zip(ratio, ratio[1:]))
    lo = math.floor(128 * math.log(4096 / (2 * math.pi * 32)) / (2 * math.log(10000)))
    hi = math.ceil(128 * math.log(4096 / (2 * math.pi)) / (2 * math.log(10000)))
    assert abs(ratio[lo] - 1) < 1e-9 < ratio[lo + 1] - 1 and ratio[hi - 1] < 16 - 1e-9 < ratio[hi]
    wide, _ = blink.blink_rope_table(128, 10000.0, scaling="base", factor=4.0, device="cpu")
    for i in (0, 1, 31, 63):
        want = (10000.0 * 4.0 ** (128 / 126)) ** (-2 * i / 128) / (2 * math.pi)
        assert abs(int(wide[i]) / 2**64 / want - 1) < 1e-13
    assert abs(int(plain[63]) / int(wide[63]) - 4) < 1e-9  # the slowest pair is stretched by the factor


@pytest.mark.parametrize("bad,status", [
    (dict(rot=0), RANGE), (dict(rot=514), RANGE), (dict(rot=63), INVALID), (dict(base=1.0), INVALID), (dict(base=NAN), INVALID),
    (dict(base=INF), INVALID), (dict(kind=5), INVALID), (dict(kind=-1), INVALID), (dict(kind=1, factor=0.5), INVALID),
    (dict(kind=1, factor=NAN), INVALID), (dict(kind=2, rot=2), INVALID), (dict(kind=2, factor=1e308, rot=4), INVALID),
    (dict(kind=3, original=0), INVALID), (dict(kind=4, low=0.0), INVALID), (dict(kind=4, low=4.0), INVALID),
    (dict(kind=3, high=INF), INVALID), (dict(turns=None), INVALID), (dict(amp=None), INVALID),
])
def test_table_refusals(lib, bad, status):
    buf, amp = (ctypes.c_uint64 * 256)(), ctypes.c_float()
    a = dict(rot=64, base=10000.0, kind=0, factor=2.0, original=4096, low=1.0, high=4.0, turns=buf, amp=ctypes.byref(amp))
    a.update(bad)
    assert lib.blink_rope_table(a["rot"], a["base"], a["kind"], a["factor"], a["original"], a["low"], a["high"], a["turns"],
                                a["amp"]) == status


QB, KB, QO, KO = 0x10000000, 0x20000000, 0x30000000, 0x40000000


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(pos=None), INVALID), (dict(turns=None), INVALID),
    (dict(k=None), INVALID), (dict(ko=None), INVALID), (dict(rows=-1), INVALID), (dict(rows=(1 << 30) + 1), RANGE),
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(d=514, qs=1 << 20, ks=1 << 20, qos=1 << 20, kos=1 << 20), RANGE),
    (dict(rot=0), INVALID), (dict(rot=65), INVALID), (dict(rot=66), INVALID), (dict(qs=255), INVALID), (dict(kos=127), INVALID),
    (dict(amp=NAN), INVALID), (dict(inter=2), INVALID),
    (dict(qo=QB + 2), INVALID), (dict(qo=QB, qos=512), INVALID), (dict(qo=KB), INVALID), (dict(ko=QB), INVALID),
    (dict(ko=QO), INVALID), (dict(qs=512, qos=512, qo=QB + 510), INVALID),  # the halves of the rows overlap by a value
])
def test_rope_refusals(lib, bad, status):
    a = dict(q=QB, qs=256, k=KB, ks=128, pos=FAKE, rows=10, Hq=4, Hkv=2, d=64, rot=64, turns=FAKE, amp=1.0, inter=0, qo=QO, qos=256,
             ko=KO, kos=128)
    a.update(bad)
    assert lib.blink_rope(_p(a["q"]), a["qs"], _p(a["k"]), a["ks"], _p(a["pos"]), a["rows"], a["Hq"], a["Hkv"], a["d"], a["rot"],
                          _p(a["turns"]), a["amp"], a["inter"], _p(a["qo"]), a["qos"], _p(a["ko"]), a["kos"], None) == status


def test_rope_of_no_rows_does_nothing(lib):
    assert lib.blink_rope(_p(QB), 256, None, 0, _p(FAKE), 0, 4, 0, 64, 64, _p(FAKE), 1.0, 0, _p(QO), 256, None, 0, None) == OK


CACHE_BAD = [(dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
             (dict(kc=FAKE + 8), INVALID), (dict(pstride=2040), INVALID), (dict(pstride=2056), INVALID), (dict(sstride=1), INVALID),
             (dict(pages=0), RANGE), (dict(page=8), INVALID), (dict(page=48), INVALID), (dict(d=96), INVALID),
             (dict(table=None), INVALID), (dict(width=0), INVALID), (dict(tstride=3), INVALID), (dict(ws=None), INVALID)]


@pytest.mark.parametrize("bad,status", CACHE_BAD + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cu=None), INVALID), (dict(start=None), INVALID), (dict(n=-1), INVALID),
    (dict(kst=120), INVALID), (dict(vst=132), INVALID), (dict(k=FAKE + 2), INVALID), (dict(S=0), RANGE), (dict(S=32769), RANGE),
    (dict(max_new=-1), INVALID), (dict(max_new=131073), RANGE), (dict(rot=66), INVALID), (dict(rot=3), INVALID), (dict(rot=-2), INVALID),
    (dict(turns=None), INVALID), (dict(amp=INF), INVALID), (dict(inter=7), INVALID), (dict(wsb=255), SMALL),
    (dict(Hkv=0), INVALID), (dict(Hkv=1025, pstride=1 << 22, sstride=2000), RANGE),
])
def test_append_refusals(lib, bad, status):
    a = dict(k=FAKE, kst=128, v=FAKE, vst=128, n=10, Hkv=2, d=64, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pstride=2048, sstride=2, pages=4,
             page=16, table=FAKE, tstride=4, width=4, cu=FAKE, start=FAKE, S=2, max_new=10, pos=None, turns=FAKE, rot=64, amp=1.0,
             inter=0, ws=FAKE, wsb=256)
    a.update(bad)
    assert lib.blink_paged_append(_p(a["k"]), a["kst"], _p(a["v"]), a["vst"], a["n"], a["Hkv"], a["d"], _p(a["kc"]), _p(a["vc"]),
                                  _p(a["ks"]), _p(a["vs"]), a["pstride"], a["sstride"], a["pages"], a["page"], _p(a["table"]),
                                  a["tstride"], a["width"], _p(a["cu"]), _p(a["start"]), a["S"], a["max_new"], _p(a["pos"]),
                                  _p(a["turns"]), a["rot"], a["amp"], a["inter"], _p(a["ws"]), a["wsb"], None) == status


@pytest.mark.parametrize("bad,status", CACHE_BAD + [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(len=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(ws=FAKE + 4), INVALID),
    (dict(S=0), RANGE), (dict(T=0), INVALID), (dict(T=65), RANGE), (dict(max_len=-1), INVALID), (dict(max_len=131073), RANGE),
    (dict(Hq=5), INVALID), (dict(Hq=258), RANGE), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(wsb=255), SMALL),
    (dict(Hkv=1024, Hq=1024 * 64, T=64, pstride=1 << 20, sstride=1024), RANGE),
])
def test_token_attention_refusals(lib, bad, status):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pstride=2048, sstride=2, pages=4, page=16, table=FAKE, tstride=4, width=4,
             len=FAKE, S=2, T=1, max_len=64, Hq=4, Hkv=2, d=64, scale=0.0, out=FAKE, lse=None, ws=FAKE, wsb=1 << 20)
    a.update(bad)
    assert lib.blink_paged_token_attention(_p(a["q"]), _p(a["kc"]), _p(a["vc"]), _p(a["ks"]), _p(a["vs"]), a["pstride"], a["sstride"],
                                           a["pages"], a["page"], _p(a["table"]), a["tstride"], a["width"], _p(a["len"]), a["S"],
                                           a["T"], a["max_len"], a["Hq"], a["Hkv"], a["d"], a["scale"], _p(a["out"]), _p(a["lse"]),
                                           _p(a["ws"]), a["wsb"], None) == status


def _c(values):
    return None if values is None else (ctypes.c_int32 * len(values))(*values)


@pytest.mark.parametrize("bad,status", CACHE_BAD + [
    (dict(q=None), INVALID), (dict(kt=None), INVALID), (dict(vt=None), INVALID), (dict(cu=None), INVALID), (dict(out=None), INVALID),
    (dict(kt=FAKE + 2), INVALID), (dict(rows=0), INVALID), (dict(B=0), RANGE), (dict(max_tail=0), INVALID),
    (dict(max_tail=131073), RANGE), (dict(n_req=0), RANGE), (dict(n_req=65, req=list(range(66)), pre=[1] * 65, rows=65), RANGE),
    (dict(req=None), INVALID), (dict(pre=None), INVALID), (dict(req=[0, 5, 9]), INVALID), (dict(req=[1, 5, 10]), INVALID),
    (dict(req=[0, 11, 10]), INVALID), (dict(pre=[64, -1]), INVALID), (dict(pre=[64, 131073]), RANGE),
    (dict(ws=FAKE + 16), INVALID),
    (dict(pre=[64, 65]), RANGE),  # more than four pages of 16 hold
    (dict(Hq=5), INVALID), (dict(Hq=258), INVALID), (dict(scale=NAN), INVALID), (dict(wsb=1000), SMALL),
])
def test_prefix_tail_refusals(lib, bad, status):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pstride=2048, sstride=2, pages=4, page=16, table=FAKE, tstride=4, width=4,
             kt=FAKE, vt=FAKE, cu=FAKE, seq=None, B=2, rows=10, n_req=2, req=[0, 5, 10], pre=[64, 10], max_tail=5, Hq=4, Hkv=2, d=64,
             scale=0.0, out=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(bad)
    assert lib.blink_paged_prefix_tail_attention(
        _p(a["q"]), _p(a["kc"]), _p(a["vc"]), _p(a["ks"]), _p(a["vs"]), a["pstride"], a["sstride"], a["pages"], a["page"],
        _p(a["table"]), a["tstride"], a["width"], _p(a["kt"]), _p(a["vt"]), _p(a["cu"]), _p(a["seq"]), a["B"], a["rows"], a["n_req"],
        _c(a["req"]), _c(a["pre"]), a["max_tail"], a["Hq"], a["Hkv"], a["d"], a["scale"], _p(a["out"]), None, _p(a["ws"]), a["wsb"],
        None) == status


def test_workspaces(lib):
    assert blink.paged_append_workspace_bytes() == 256
    one = blink.paged_token_attention_workspace_bytes(1, 1, 100, 4, 2, 64)
    assert one >= 256
    assert blink.paged_token_attention_workspace_bytes(8, 1, 131072, 32, 8, 128) > one
    assert lib.blink_paged_token_attention_workspace(0, 1, 10, 4, 2, 64) == 256  # refused by the call itself
    # many tail rows: the prefixes' rows in whole key tiles, K and V, 2 bytes a value; few rows: less
    assert blink.paged_prefix_tail_workspace_bytes([0, 500, 1000], [1, 129], 2, 4, 2, 64) >= (128 + 256) * 2 * 64 * 2 * 2
    assert blink.paged_prefix_tail_workspace_bytes([0, 1, 2], [1, 131072], 2, 4, 2, 64) < 131072 * 2 * 64 * 2 * 2
    with pytest.raises(ValueError):
        blink.paged_prefix_tail_workspace_bytes([0, 5], [1, 129], 2, 4, 2, 64)


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        blink.blink_rope(q, None, i32, torch.zeros(32, dtype=torch.int64))
    cache = blink.blink_paged_cache(2, 16, 4, 64, device="cpu")
    assert cache["k"].dtype == torch.float8_e4m3fn and cache["k"].shape == (2, 4, 16, 64) and cache["v_scale"].shape == (2, 4)
    with pytest.raises(ValueError, match="CUDA"):
        blink.blink_paged_append(q, q, cache, torch.zeros(1, 2, dtype=torch.int32), i32[:2], i32[:1], 3)
    with pytest.raises(ValueError, match="CUDA"):
        blink.blink_paged_token_attention(q.view(3, 1, 4, 64), cache, torch.zeros(3, 2, dtype=torch.int32), i32, 10)
    with pytest.raises(ValueError, match="CUDA"):
        blink.blink_paged_prefix_tail_attention(q, cache, torch.zeros(1, 2, dtype=torch.int32), [5], q, q, i32[:2], 1, 3)
    with pytest.raises(ValueError, match="scaling"):
        blink.blink_rope_table(64, scaling="other", device="cpu")
    with pytest.raises(blink.BlinkError):
        blink.blink_rope_table(63, device="cpu")
