"""Rotary positions against the plain form in 64 bits: layouts, partial rotation, scalings, far and negative
positions, strides and alignments, in place, on another stream."""
import pytest
import torch

from shared_prefix_question_gb300 import blink

pytestmark = pytest.mark.gpu
from tests import paged_helpers as ph  # noqa: E402


def _check(got, x, pos, theta, amplitude, interleaved):
    want, size = ph.rotate(x, pos, theta, amplitude, interleaved)
    # the angle's and the functions' errors and three products' roundings in 32 bits, then one to bf16
    bound = ph.BF16 * want.abs() + 8 * ph.F32 * size + 2.0 ** -133
    rot = 2 * len(theta)
    assert bool(((got.double() - want).abs() <= bound)[..., :rot].all())
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("rows,Hq,Hkv,d,rot", [(1, 32, 8, 128, 128), (7, 4, 2, 64, 64), (65, 5, 1, 64, 32), (33, 3, 2, 80, 20),
                                               (9, 28, 4, 128, 2), (1300, 32, 8, 128, 64), (3, 1, 1, 512, 512), (2, 2, 1, 6, 4),
                                               (640, 8, 8, 128, 120), (11, 2, 2, 72, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_sizes(rows, Hq, Hkv, d, rot, interleaved):
    g = ph.gen(rows + d)
    q, k = (ph.randn(g, rows, H, d).to(torch.bfloat16) for H in (Hq, Hkv))
    pos = torch.randint(0, 131072, (rows,), device="cuda", generator=g).to(torch.int32)
    turns, amplitude = blink.blink_rope_table(rot, 10000.0)
    theta, _ = ph.frequencies(rot, 10000.0)
    qo, ko = blink.blink_rope(q, k, pos, turns, interleaved=interleaved, amplitude=amplitude)
    _check(qo, q, pos, theta, 1.0, interleaved)
    _check(ko, k, pos, theta, 1.0, interleaved)
    q1, none = blink.blink_rope(q, None, pos, turns, interleaved=interleaved)
    assert none is None and torch.equal(q1, qo)


@pytest.mark.parametrize("scaling,args", [(None, {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                          ("by_dim", dict(factor=8.0, original=4096, low=1.0, high=32.0)),
                                          ("by_turns", dict(factor=8.0, original=8192, low=1.0, high=4.0))])
@pytest.mark.parametrize("amp", [1.0, 0.5])
def test_rope_scalings_and_far_positions(scaling, args, amp):
    g = ph.gen(5)
    pos = torch.tensor([0, 1, -1, 17, 131071, -131071, 1 << 20, 2**31 - 1, -2**31], dtype=torch.int32, device="cuda")
    q = ph.randn(g, len(pos), 2, 128).to(torch.bfloat16)
    turns, amplitude = blink.blink_rope_table(128, 500000.0, scaling=scaling, **args)
    theta, want = ph.frequencies(128, 500000.0, scaling, **args)
    assert abs(amplitude - want) <= 2.0 ** -24 * want
    out, _ = blink.blink_rope(q, None, pos, turns, amplitude=amplitude * amp)
    near = pos.abs() <= 1 << 20
    near[-1] = False
    _check(out[near], q[near], pos[near], theta, amplitude * amp, False)
    # at 2^31 the table's 53 bits leave 2^-25 turns, 2^-22 radians
    w, size = ph.rotate(q, pos, theta, amplitude * amp, False)
    assert bool(((out.double() - w).abs() <= ph.BF16 * w.abs() + (2.0 ** -21 + 8 * ph.F32) * size + 2.0 ** -133).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,shift", [(128, 128, 0), (64, 40, 0), (128, 64, 4), (64, 64, 1)])
def test_rope_slices_of_one_projection_in_place(interleaved, d, rot, shift):
    """Rows of q, k, v side by side, at an offset that may not be 16-byte aligned; v and the pad stay as they are."""
    g = ph.gen(d + rot)
    rows, Hq, Hkv = 37, 4, 2
    wide = (Hq + 2 * Hkv) * d + 8
    flat = ph.randn(g, rows * wide + shift).to(torch.bfloat16)
    row = flat[shift:].view(rows, wide)
    before = row.clone()
    q, k = row[:, :Hq * d].view(rows, Hq, d), row[:, Hq * d:(Hq + Hkv) * d].view(rows, Hkv, d)
    q0, k0 = q.clone(), k.clone()
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") * 1000
    turns, _ = blink.blink_rope_table(rot)
    theta, _ = ph.frequencies(rot, 10000.0)
    want_q, want_k = blink.blink_rope(q0, k0, pos, turns, interleaved=interleaved)
    blink.blink_rope(q, k, pos, turns, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    _check(q, q0, pos, theta, 1.0, interleaved)
    assert torch.equal(row[:, (Hq + Hkv) * d:], before[:, (Hq + Hkv) * d:])


def test_rope_there_and_back():
    """Keys moved by -p return to where they were, within the two roundings."""
    g = ph.gen(1)
    k = ph.randn(g, 50, 8, 128).to(torch.bfloat16)
    pos = torch.randint(0, 100000, (50,), device="cuda", generator=g).to(torch.int32)
    turns, _ = blink.blink_rope_table(128)
    there, _ = blink.blink_rope(k, None, pos, turns)
    back, _ = blink.blink_rope(there, None, -pos, turns)
    size = torch.cat([k[..., :64].abs() + k[..., 64:].abs()] * 2, dim=-1).double()
    assert bool(((back.double() - k.double()).abs() <= ph.BF16 * k.double().abs() + (ph.BF16 * 1.5 + 16 * ph.F32) * size).all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_values_past_rot_pass_whatever_they_hold(interleaved):
    x = torch.ones(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    x[..., 20:] = float("nan")
    x[..., 40:] = float("inf")
    turns, _ = blink.blink_rope_table(20)
    out, _ = blink.blink_rope(x, None, torch.tensor([0, 3, 9], dtype=torch.int32, device="cuda"), turns, interleaved=interleaved)
    assert bool(out[..., :20].isfinite().all()) and torch.equal(out[..., 20:].isnan(), x[..., 20:].isnan())
    assert torch.equal(out[..., 40:], x[..., 40:])


def test_rope_no_rows_another_stream_and_capture():
    turns, _ = blink.blink_rope_table(64)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, k = blink.blink_rope(q, q, torch.empty(0, dtype=torch.int32, device="cuda"), turns)
    assert out.shape == k.shape == (0, 4, 64)
    g = ph.gen(2)
    q = ph.randn(g, 40, 4, 64).to(torch.bfloat16)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    want, _ = blink.blink_rope(q, None, pos, turns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = blink.blink_rope(q, None, pos, turns, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    into = torch.empty_like(q)
    with torch.cuda.graph(graph):
        blink.blink_rope(q, None, pos, turns, q_out=into)
    pos += 5
    graph.replay()
    assert torch.equal(into, blink.blink_rope(q, None, pos, turns)[0])
