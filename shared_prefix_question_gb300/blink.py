"""Thin Python binding of the C ABI in include/blink.h (libblink.so, built in-tree for sm_103a).

Argument marshalling only: every step of the path runs in the library's CUDA kernels.  Torch
tensors supply device memory and the current CUDA stream; outputs are allocated with torch when
the caller does not pass them.  There is no CPU fallback: without the built library or a CUDA
device every call raises.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libblink.so")

BLINK_OK = 0
BLINK_INVALID_ARG = 1
BLINK_OUT_OF_RANGE = 2
BLINK_WORKSPACE_TOO_SMALL = 3
BLINK_CUDA_ERROR = 4
BLINK_DEVICE_FLAG = 5
BLINK_DEVICE_TIMEOUT = 6

MAX_OPTIONS = 255
MAX_QUESTIONS = 512
MAX_INPUT_TOKENS = 131072
MAX_PLAN_SEQUENCES = 32768
MAX_TOP_TOKENS = 32


class BlinkError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lib = None

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_f32 = ctypes.c_float
_f64 = ctypes.c_double
_sz = ctypes.c_size_t

_SIGNATURES = {
    "blink_status_string": (ctypes.c_char_p, [_i32]),
    "blink_read_device_status": (_i32, [_vp, _i32, _vp]),
    "blink_selftest_wait_timeout": (_i32, [ctypes.c_uint32, _vp, _sz, _vp]),
    "blink_pack_plan_workspace": (_sz, [_i32]),
    "blink_pack_plan": (_i32, [_vp, _i32, _i32, _i32] + [_vp] * 10 + [_vp]),
    "blink_attention_workspace": (_sz, [_i32] * 6),
    "blink_attention_split_plan": (_i32, [_i32] * 6 + [_vp] * 3),
    "blink_prefix_tail_attention": (_i32, [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                           _i32, _i32, _f32, _vp, _vp, _vp, _sz, _vp]),
    "blink_prefix_tail_attention_multi": (_i32, [_vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp,
                                                 _vp, _vp, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _vp, _sz, _vp]),
    "blink_shared_prefix_len_workspace": (_sz, []),
    "blink_shared_prefix_len": (_i32, [_vp, _i64, _vp, _i32, _vp, _vp, _vp, _sz, _vp]),
    "blink_kv_to_arena": (_i32, [_vp, _vp, _i64, _i64, _i32, _vp, _vp, _i64, _i64, _i64, _vp]),
    "blink_rotation_debias_workspace": (_sz, []),
    "blink_rotation_debias": (_i32, [_vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _f32, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _vp, _sz, _vp]),
    "blink_label_readout_workspace": (_sz, [_i32]),
    "blink_label_readout": (_i32, [_vp, _i64, _i32, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _i32, _i32, _f32, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _vp, _sz, _vp]),
    "blink_label_readout_noalloc": (_i32, [_vp, _i64, _i32, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _i32, _i32, _f32, _vp,
                                           _vp, _vp, _vp]),
    "blink_prefix_key_weights_workspace": (_sz, [_i32] * 5),
    "blink_prefix_key_weights": (_i32, [_vp, _vp, _i64, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _f32, _f32, _vp, _i64,
                                        _vp, _i64, _vp, _sz, _vp]),
    "blink_kv_evict_workspace": (_sz, [_i32] * 3),
    "blink_kv_evict": (_i32, [_vp, _i64, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _i64, _vp, _vp, _i64,
                              _vp, _vp, _i64, _vp, _i64, _vp, _sz, _vp]),
    "blink_token_logprobs_workspace": (_sz, [_i32] * 4),
    "blink_token_logprobs_workspace_plan": (_i32, [_i32] * 5 + [_vp, _vp]),
    "blink_token_logprobs": (_i32, [_vp, _i64, _i32, _vp, _vp, _i32, _i32, _vp, _i32, _f32, _i32] + [_vp] * 6 +
                             [_sz, _vp]),
    "blink_rope_table": (_i32, [_i32, _f64, _i32, _f64, _i32, _f64, _f64, _vp, _vp]),
    "blink_rope": (_i32, [_vp, _i64, _vp, _i64, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _f32, _i32, _vp, _i64, _vp, _i64, _vp]),
    "blink_paged_append_workspace": (_sz, []),
    "blink_paged_append": (_i32, [_vp, _i64, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _i64,
                                  _i32, _vp, _vp, _i32, _i32, _vp, _vp, _i32, _f32, _i32, _vp, _sz, _vp]),
    "blink_paged_token_attention_workspace": (_sz, [_i32] * 6),
    "blink_paged_token_attention": (_i32, [_vp] * 5 + [_i64, _i64, _i32, _i32, _vp, _i64, _i32, _vp, _i32, _i32, _i32, _i32,
                                                       _i32, _i32, _f32, _vp, _vp, _vp, _sz, _vp]),
    "blink_paged_prefix_tail_workspace": (_sz, [_vp, _vp, _i32, _i32, _i32, _i32, _i32]),
    "blink_paged_prefix_tail_attention": (_i32, [_vp] * 5 + [_i64, _i64, _i32, _i32, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _i32,
                                                             _i32, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _vp,
                                                             _sz, _vp]),
}


def lib():
    """Load libblink.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() or "
                               "python -m shared_prefix_question_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return list(_SIGNATURES)


def status_string(status: int) -> str:
    try:
        return lib().blink_status_string(int(status)).decode()
    except Exception:  # library not loadable: still give a readable message
        return "status"


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: torch.cuda.Stream | None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors passed to the library must be contiguous CUDA tensors")


def _check(status: int, what: str):
    if status != BLINK_OK:
        raise BlinkError(status, what)


# ------------------------------------------------------------------------------------------------ plan
def blink_pack_plan(lengths: torch.Tensor, budget: int, max_rows: int = 0, out: dict | None = None,
                    sync: bool = False, stream=None) -> dict:
    """Token-budget pack plan of int32 `lengths` (device).  Returns the plan tensors; with
    sync=True also `n_forwards` as a Python int (one pinned D2H copy, synchronising)."""
    _need_cuda(lengths)
    if lengths.dtype != torch.int32:
        raise ValueError("lengths must be int32")
    n = lengths.numel()
    dev = lengths.device
    if out is None:
        out = {k: torch.empty(n + (1 if k in ("fwd_slot_start", "cu_seqlens") else 0), dtype=torch.int32, device=dev)
               for k in ("order", "slot_of", "fwd_of_slot", "fwd_slot_start", "fwd_width", "cu_seqlens",
                         "last_varlen", "last_padded")}
        out["n_forwards_dev"] = torch.empty(1, dtype=torch.int32, device=dev)
    host = torch.empty(1, dtype=torch.int32, pin_memory=True) if sync else None
    st = lib().blink_pack_plan(_ptr(lengths), n, int(budget), int(max_rows), _ptr(out["order"]),
                               _ptr(out["slot_of"]), _ptr(out["fwd_of_slot"]), _ptr(out["fwd_slot_start"]), _ptr(out["fwd_width"]),
                               _ptr(out["cu_seqlens"]), _ptr(out["last_varlen"]), _ptr(out["last_padded"]),
                               _ptr(out["n_forwards_dev"]), _ptr(host), _stream(stream))
    _check(st, "blink_pack_plan")
    if sync:
        out["n_forwards"] = int(host.item())
    return out


# ------------------------------------------------------------------------------------------------ attention
def pack_plan_workspace_bytes(n: int) -> int:
    """0: the planner's scratch is its own output arrays."""
    return int(lib().blink_pack_plan_workspace(n))


def attention_workspace_bytes(rows, B, P, Hq, Hkv, d) -> int:
    return int(lib().blink_attention_workspace(rows, B, P, Hq, Hkv, d))


def blink_attention_split_plan(rows: int, P: int, Hq: int, Hkv: int, d: int, sms: int):
    """The prefix-chunk plan of one request on a GPU with `sms` SMs (host computation only):
    (whole_units, chunks, chunk_tiles) as include/blink.h describes them."""
    w, c, t = ctypes.c_int64(0), ctypes.c_int32(0), ctypes.c_int32(0)
    st = lib().blink_attention_split_plan(int(rows), int(P), int(Hq), int(Hkv), int(d), int(sms), ctypes.byref(w),
                                          ctypes.byref(c), ctypes.byref(t))
    _check(st, "blink_attention_split_plan")
    return int(w.value), int(c.value), int(t.value)


def new_workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled device workspace (the first word is the device error word)."""
    return torch.zeros(max(256, (nbytes + 255) // 256 * 256), dtype=torch.uint8, device=device)


def blink_prefix_tail_attention(q, k_pre, v_pre, k_tail, v_tail, cu_seqlens, B: int, P: int, max_tail: int,
                                seq_start=None, scale: float = 0.0, out=None, lse=None, want_lse: bool = False,
                                ws=None, pre_row_stride: int | None = None, stream=None):
    """q [rows, Hq, d], k_tail/v_tail [rows, Hkv, d], k_pre/v_pre [P, Hkv, d] (or rows of an arena with
    `pre_row_stride` elements), all bf16 on the device.  Returns (out, lse, ws)."""
    _need_cuda(q, k_tail, v_tail, cu_seqlens, seq_start)
    rows, Hq, d = q.shape
    Hkv = k_tail.shape[1]
    if P > 0:
        if pre_row_stride is None:
            _need_cuda(k_pre, v_pre)
            pre_row_stride = Hkv * d
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(Hq, rows, dtype=torch.float32, device=q.device)
    need = attention_workspace_bytes(rows, B, P, Hq, Hkv, d)
    if ws is None:
        ws = new_workspace(need, q.device)
    st = lib().blink_prefix_tail_attention(
        _ptr(q), _ptr(k_pre) if P > 0 else None, _ptr(v_pre) if P > 0 else None, int(pre_row_stride or 0),
        _ptr(k_tail), _ptr(v_tail), _ptr(cu_seqlens), _ptr(seq_start), int(B), int(rows), int(P), int(max_tail),
        int(Hq), int(Hkv), int(d), float(scale), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "blink_prefix_tail_attention")
    return out, lse, ws


def blink_prefix_tail_attention_multi(q, k_arena, v_arena, k_tail, v_tail, cu_seqlens, B: int, req_rows,
                                      req_prefix_start, req_prefix_len, max_tail: int, seq_start=None,
                                      scale: float = 0.0, out=None, lse=None, want_lse: bool = False, ws=None,
                                      arena_row_stride: int | None = None, stream=None):
    """Several requests in one launch: request r owns rows [req_rows[r], req_rows[r+1]) of q/k_tail/
    v_tail and attends to arena slots [req_prefix_start[r], + req_prefix_len[r]).  The arena tensors
    are [slots, Hkv, d] (or [slots, stride] with `arena_row_stride`).  Returns (out, lse, ws)."""
    import numpy as np
    _need_cuda(q, k_tail, v_tail, cu_seqlens, seq_start)
    rows, Hq, d = q.shape
    Hkv = k_tail.shape[1]
    n_req = len(req_prefix_len)
    h_rows = np.ascontiguousarray(req_rows, dtype=np.int32)
    h_start = np.ascontiguousarray(req_prefix_start, dtype=np.int32)
    h_len = np.ascontiguousarray(req_prefix_len, dtype=np.int32)
    if arena_row_stride is None:
        arena_row_stride = Hkv * d
    slots = int(k_arena.shape[0]) if k_arena is not None else 0
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(Hq, rows, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = new_workspace(attention_workspace_bytes(rows, B, 0, Hq, Hkv, d), q.device)
    st = lib().blink_prefix_tail_attention_multi(
        _ptr(q), _ptr(k_arena), _ptr(v_arena), int(arena_row_stride), slots,
        _ptr(k_tail), _ptr(v_tail), _ptr(cu_seqlens), _ptr(seq_start), int(B), int(rows), int(n_req),
        h_rows.ctypes.data_as(ctypes.c_void_p), h_start.ctypes.data_as(ctypes.c_void_p),
        h_len.ctypes.data_as(ctypes.c_void_p), int(max_tail), int(Hq), int(Hkv), int(d), float(scale), _ptr(out),
        _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "blink_prefix_tail_attention_multi")
    return out, lse, ws


def blink_read_device_status(ws: torch.Tensor, clear: bool = True, stream=None) -> int:
    return int(lib().blink_read_device_status(_ptr(ws), 1 if clear else 0, _stream(stream)))


def blink_selftest_wait_timeout(limit_us: int, ws: torch.Tensor, stream=None) -> int:
    """Runs the bounded device wait against a barrier nothing arrives at; returns the status it
    latched (BLINK_DEVICE_TIMEOUT when the failure path works)."""
    return int(lib().blink_selftest_wait_timeout(int(limit_us), _ptr(ws), ws.numel(), _stream(stream)))


# ------------------------------------------------------------------------------------------------ readout
def readout_workspace_bytes(B: int) -> int:
    return int(lib().blink_label_readout_workspace(B))


def blink_label_readout(hidden, last_idx, unembed, label_off, label_ids, temperature: float, probs=None,
                        host_probs=None, logits=None, ws=None, slot_of=None, qtype=None, answers=None,
                        host_answers=None, stream=None):
    """hidden [rows, H] bf16, last_idx int32 (per question, or per slot with `slot_of`), unembed [V, H]
    bf16, CSR label_off [B+1] / label_ids [sum K] int32, all on the device.  Returns (probs, ws); if
    `host_probs` (pinned fp32) is given the call copies into it and synchronises."""
    _need_cuda(hidden, last_idx, unembed, label_off, label_ids, probs, logits, slot_of, qtype, answers)
    rows, H = hidden.shape
    V = unembed.shape[0]
    B = label_off.numel() - 1
    sum_k = label_ids.numel()
    if probs is None:
        probs = torch.empty(sum_k, dtype=torch.float32, device=hidden.device)
    if qtype is not None and answers is None:
        answers = torch.empty(B, 3, dtype=torch.float32, device=hidden.device)
    if ws is None:
        ws = new_workspace(readout_workspace_bytes(B), hidden.device)
    st = lib().blink_label_readout(_ptr(hidden), int(hidden.stride(0)), int(rows), _ptr(last_idx), _ptr(slot_of), _ptr(unembed),
                                   int(V), int(H), _ptr(label_off), _ptr(label_ids), int(B), int(sum_k),
                                   float(temperature), _ptr(probs), _ptr(host_probs), _ptr(logits), _ptr(qtype),
                                   _ptr(answers), _ptr(host_answers), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "blink_label_readout")
    if answers is not None:
        return probs, ws, answers
    return probs, ws


STATIC_SCRATCH_QUESTIONS = 32768


def blink_label_readout_noalloc(hidden, last_idx, unembed, label_off, label_ids, temperature: float, probs=None,
                                host_probs=None, logits=None, slot_of=None, stream=None):
    """The readout for callers that cannot allocate device memory (the library keeps its scratch in a
    static device array; at most 32768 questions; calls that overlap on the GPU race).  Outputs are
    allocated here only when the caller passes none.

    Device-side errors (a label id outside [0, V), malformed offsets) are reported only when
    `host_probs` is given: the C call then reads the error word back after its copy and this
    wrapper raises BlinkError.  Without `host_probs` the call stays asynchronous and such a
    question's probabilities come back as NaN (or, for malformed offsets, unwritten)."""
    _need_cuda(hidden, last_idx, unembed, label_off, label_ids, probs, logits, slot_of)
    rows, H = hidden.shape
    V = unembed.shape[0]
    B = label_off.numel() - 1
    sum_k = label_ids.numel()
    if probs is None:
        probs = torch.empty(sum_k, dtype=torch.float32, device=hidden.device)
    st = lib().blink_label_readout_noalloc(_ptr(hidden), int(hidden.stride(0)), int(rows), _ptr(last_idx),
                                           _ptr(slot_of), _ptr(unembed), int(V), int(H), _ptr(label_off),
                                           _ptr(label_ids), int(B), int(sum_k), float(temperature), _ptr(probs),
                                           _ptr(host_probs), _ptr(logits), _stream(stream))
    _check(st, "blink_label_readout_noalloc")
    return probs


# ------------------------------------------------------------------------------------------------ prefix side
def blink_shared_prefix_len(tokens, cu, out=None, sync: bool = True, ws=None, stream=None):
    """Shared-prefix length of the sequences in `tokens` (int32, back to back, offsets `cu`)."""
    _need_cuda(tokens, cu)
    n = cu.numel() - 1
    if out is None:
        out = torch.empty(1, dtype=torch.int32, device=tokens.device)
    if ws is None:
        ws = new_workspace(int(lib().blink_shared_prefix_len_workspace()), tokens.device)
    host = torch.empty(1, dtype=torch.int32, pin_memory=True) if sync else None
    st = lib().blink_shared_prefix_len(_ptr(tokens), int(tokens.numel()), _ptr(cu), int(n), _ptr(out), _ptr(host),
                                       _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "blink_shared_prefix_len")
    return int(host.item()) if sync else out


def blink_kv_to_arena(k_src, v_src, k_arena, v_arena, dst_slot: int, stream=None):
    """Write the token rows of k_src / v_src ([n, ...] bf16, rows contiguous) into arena rows
    [dst_slot, dst_slot + n) of k_arena / v_arena ([slots, stride] bf16)."""
    n = k_src.shape[0]
    row_elems = k_src[0].numel() if n else 0
    st = lib().blink_kv_to_arena(_ptr(k_src), _ptr(v_src), int(k_src.stride(0)), int(n), int(row_elems),
                                 _ptr(k_arena), _ptr(v_arena), int(k_arena.stride(0)), int(k_arena.shape[0]),
                                 int(dst_slot), _stream(stream))
    _check(st, "blink_kv_to_arena")


def blink_rotation_debias(logits, pass_off, key_of_pos, question_pass, raw_off, temperature: float, prior=None,
                          raw=None, probs=None, host_probs=None, qtype=None, answers=None, host_answers=None,
                          ws=None, sum_k: int | None = None, stream=None):
    """Per pass log-softmax minus the prior, the mean over each question's passes, then the
    temperature softmax (and optional typed answers).  Returns (probs, raw, answers)."""
    _need_cuda(logits, pass_off, key_of_pos, question_pass, raw_off, prior, raw, probs, qtype, answers)
    n_pass = pass_off.numel() - 1
    B = raw_off.numel() - 1
    if sum_k is None:
        sum_k = int(raw_off[-1].item())  # one small copy; pass sum_k to avoid it
    dev = logits.device
    if probs is None:
        probs = torch.empty(sum_k, dtype=torch.float32, device=dev)
    if raw is None:
        raw = torch.empty(sum_k, dtype=torch.float32, device=dev)
    if qtype is not None and answers is None:
        answers = torch.empty(B, 3, dtype=torch.float32, device=dev)
    if ws is None:
        ws = new_workspace(int(lib().blink_rotation_debias_workspace()), dev)
    st = lib().blink_rotation_debias(_ptr(logits), _ptr(pass_off), _ptr(key_of_pos), int(n_pass), _ptr(question_pass),
                                     _ptr(raw_off), int(B), sum_k, _ptr(prior), float(temperature), _ptr(raw),
                                     _ptr(probs), _ptr(host_probs), _ptr(qtype), _ptr(answers), _ptr(host_answers),
                                     _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "blink_rotation_debias")
    return probs, raw, answers


# ------------------------------------------------------------------------------------------------ cache eviction
INT32_MAX = 2**31 - 1


def _refuse(name, t, dtype, shape, inner):
    """Raises what is wrong with `t` (see _need)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and w != s for w, s in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    want = 1
    for s, st in list(zip(t.shape, t.stride()))[::-1][:inner]:
        if s != 1 and st != want:
            raise ValueError(f"{name}: the last {inner} dimension(s) must be contiguous")
        want *= s


def _need(name, t, dtype, shape, inner: int = 1):
    """`t` is a CUDA tensor of `dtype` and `shape` (None leaves a size free) whose last `inner`
    dimensions are contiguous."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _refuse(name, t, dtype, shape, inner)


def _int32(name, x) -> int:
    """`x` for a 32-bit argument: ctypes would drop the bits above without a word."""
    x = operator.index(x)
    if not -INT32_MAX - 1 <= x <= INT32_MAX:
        raise ValueError(f"{name} must fit 32 bits, not {x}")
    return x


def _sizes(*sizes):
    """Sizes of tensors, passed in 32 bits."""
    if max(sizes) > INT32_MAX:
        raise ValueError(f"sizes must fit 32 bits: {max(sizes)}")


def _row_stride(t) -> int:
    """Elements between the rows (first dimension) of `t`; a single row has any stride."""
    return t[0].numel() if t.shape[0] == 1 else t.stride(0)


def _addr(t):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the current stream's handle, without an object


class _Launch:
    """The device of the call's tensors made current and its stream: `stream`, or that device's
    current one.  What the call allocates belongs to that stream, and its inputs are marked as used on
    it, so a caller that passes another stream than its tensors' own may drop them after the call."""

    __slots__ = ("device", "handle", "_contexts")

    def __init__(self, stream, first, *others):
        index = first.get_device()
        for t in others:
            if t is not None and t.get_device() != index:
                raise ValueError("tensors passed to one call must be on one device")
        self.device = first.device
        self._contexts = None
        if stream is None and index == torch.cuda.current_device():
            self.handle = _raw_stream(index) if _raw_stream else torch.cuda.current_stream().cuda_stream
            return
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        elif stream.device != self.device:
            raise ValueError("the stream belongs to another device than the tensors")
        else:
            with torch.cuda.stream(stream):
                capturing = torch.cuda.is_current_stream_capturing()
            for t in () if capturing else (first, *others):
                if t is not None:
                    t.record_stream(stream)
        self.handle = stream.cuda_stream
        self._contexts = (torch.cuda.device(self.device), torch.cuda.stream(stream))

    def __enter__(self):
        for c in self._contexts or ():
            c.__enter__()
        return self

    def __exit__(self, *exc):
        for c in reversed(self._contexts or ()):
            c.__exit__(*exc)

    def empty(self, dtype, *shape):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, nbytes: int):
        """A new workspace whose header (all that has to start at zero) is cleared."""
        ws = self.empty(torch.uint8, max(256, (nbytes + 255) // 256 * 256))
        ws[:256].zero_()
        return ws


def key_weights_workspace_bytes(rows, P, Hq, Hkv, d) -> int:
    return int(lib().blink_prefix_key_weights_workspace(int(rows), int(P), int(Hq), int(Hkv), int(d)))


def blink_prefix_key_weights(q, k_pre, lse, prev=None, decay: float = 0.0, scale: float = 0.0, out=None, ws=None,
                             stream=None):
    """Attention weight each prefix key received: q [rows, Hq, d] and k_pre [P, Hkv, d] bf16 (the rows
    of k_pre may be strided: an arena region), lse [Hq, rows] fp32 from blink_prefix_tail_attention
    (a slice of a wider one is fine).  Returns (weights [Hkv, P] fp32, ws); with `prev` and `decay` > 0
    decay * prev is added (`out=prev` accumulates in place)."""
    _need("q", q, torch.bfloat16, q.shape if getattr(q, "ndim", 0) == 3 else (None,) * 3, inner=3)
    rows, Hq, d = q.shape
    P, Hkv = k_pre.shape[:2] if getattr(k_pre, "ndim", 0) == 3 else (None, None)
    _need("k_pre", k_pre, torch.bfloat16, (P, Hkv, d), inner=2)
    _need("lse", lse, torch.float32, (Hq, rows))
    _sizes(rows, P, Hq, Hkv)
    if prev is not None:
        _need("prev", prev, torch.float32, (Hkv, P))
    if out is not None:
        _need("out", out, torch.float32, (Hkv, P))
    if ws is not None:
        _need("ws", ws, torch.uint8, (ws.numel(),))
    with _Launch(stream, q, k_pre, lse, prev, out, ws) as call:
        if out is None:
            out = call.empty(torch.float32, Hkv, P)
        if ws is None:
            ws = call.workspace(key_weights_workspace_bytes(rows, P, Hq, Hkv, d))
        st = lib().blink_prefix_key_weights(
            q.data_ptr(), k_pre.data_ptr(), _row_stride(k_pre) if P else 0, lse.data_ptr(), _row_stride(lse), rows, P, Hq, Hkv,
            d, scale, decay, _addr(prev), 0 if prev is None else _row_stride(prev), out.data_ptr(), _row_stride(out),
            ws.data_ptr(), ws.numel(), call.handle)
    _check(st, "blink_prefix_key_weights")
    return out, ws


def kv_evict_workspace_bytes(P, keep, Hkv) -> int:
    return int(lib().blink_kv_evict_workspace(int(P), int(keep), int(Hkv)))


def blink_kv_evict(weights, k, v, keep: int, pos=None, sink: int = 0, recent_from: int | None = None, k_dst=None,
                   v_dst=None, weights_dst=None, pos_dst=None, slots=None, ws=None, stream=None) -> dict:
    """Keep the `keep` heaviest of the P keys of every kv head: weights [Hkv, P] fp32, k and v
    [P, Hkv, d] bf16 arena regions (strided rows are fine), pos [Hkv, P] int32 positions (None: the slots).
    Without k_dst / v_dst the regions are compacted in place into their first `keep` rows; with them the
    kept rows are written there.  weights_dst / pos_dst may be views of weights / pos (in place).
    Returns {"slots", "k", "v", "weights", "pos", "ws"}, all of `keep` keys per head."""
    Hkv, P = weights.shape if getattr(weights, "ndim", 0) == 2 else (None, None)
    _need("weights", weights, torch.float32, (Hkv, P))
    d = k.shape[2] if getattr(k, "ndim", 0) == 3 else None
    _need("k", k, torch.bfloat16, (P, Hkv, d), inner=2)
    _need("v", v, torch.bfloat16, (P, Hkv, d), inner=2)
    keep = int(keep)
    if not 1 <= keep <= P:
        raise ValueError(f"keep must be in 1..{P}, not {keep}")
    _sizes(P, Hkv, d)
    sink = _int32("sink", sink)
    recent_from = INT32_MAX if recent_from is None else _int32("recent_from", recent_from)
    if pos is not None:
        _need("pos", pos, torch.int32, (Hkv, P))
    if (k_dst is None) != (v_dst is None):
        raise ValueError("k_dst and v_dst go together")
    src_stride = _row_stride(k)
    if P > 1 and v.stride(0) != src_stride:
        raise ValueError("k and v must have the same row stride")
    in_place = k_dst is None
    if in_place:
        k_dst, v_dst, dst_stride = k[:keep], v[:keep], src_stride
    else:
        _need("k_dst", k_dst, torch.bfloat16, (keep, Hkv, d), inner=2)
        _need("v_dst", v_dst, torch.bfloat16, (keep, Hkv, d), inner=2)
        dst_stride = _row_stride(k_dst) if keep > 1 else src_stride  # one row: so that it may be row 0 of k
        if keep > 1 and v_dst.stride(0) != dst_stride:
            raise ValueError("k_dst and v_dst must have the same row stride")
    if weights_dst is not None:
        _need("weights_dst", weights_dst, torch.float32, (Hkv, keep))
    if pos_dst is not None:
        _need("pos_dst", pos_dst, torch.int32, (Hkv, keep))
    if slots is not None:
        _need("slots", slots, torch.int32, (Hkv, keep), inner=2)
    if ws is not None:
        _need("ws", ws, torch.uint8, (ws.numel(),))
    with _Launch(stream, weights, k, v, pos, k_dst, v_dst, weights_dst, pos_dst, slots, ws) as call:
        if slots is None:
            slots = call.empty(torch.int32, Hkv, keep)
        if weights_dst is None:
            weights_dst = call.empty(torch.float32, Hkv, keep)
        if pos_dst is None:
            pos_dst = call.empty(torch.int32, Hkv, keep)
        if ws is None:
            ws = call.workspace(kv_evict_workspace_bytes(P, keep, Hkv))
        st = lib().blink_kv_evict(
            weights.data_ptr(), _row_stride(weights), _addr(pos), 0 if pos is None else _row_stride(pos), P, keep, sink,
            recent_from, Hkv, d, k.data_ptr(), v.data_ptr(), src_stride,
            k_dst.data_ptr(), v_dst.data_ptr(), dst_stride, slots.data_ptr(), weights_dst.data_ptr(), _row_stride(weights_dst),
            pos_dst.data_ptr(), _row_stride(pos_dst), ws.data_ptr(), ws.numel(), call.handle)
    _check(st, "blink_kv_evict")
    return {"slots": slots, "k": k_dst, "v": v_dst, "weights": weights_dst, "pos": pos_dst, "ws": ws}


# ------------------------------------------------------------------------------------------------ whole vocabulary
def token_logprobs_workspace_bytes(n, H, V, top) -> int:
    return int(lib().blink_token_logprobs_workspace(int(n), int(H), int(V), int(top)))


def blink_token_logprobs_workspace_plan(n: int, H: int, V: int, top: int, sms: int):
    """(bytes of the workspace, most bytes a launch of the call lays out) on a GPU with `sms` SMs (host
    computation only)."""
    ws, used = ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = lib().blink_token_logprobs_workspace_plan(int(n), int(H), int(V), int(top), int(sms), ctypes.byref(ws),
                                                   ctypes.byref(used))
    _check(st, "blink_token_logprobs_workspace_plan")
    return int(ws.value), int(used.value)


def blink_token_logprobs(hidden, unembed, targets=None, row_idx=None, temperature: float = 1.0, top: int = 0, ws=None,
                         stream=None) -> dict:
    """Whole-vocabulary readout of hidden rows [rows, H] bf16 (all of them, or those of int32 `row_idx`)
    against unembed [V, H] bf16.  Returns {"logprob" (of int32 `targets`, else None), "entropy", "lse",
    "top_ids", "top_logprobs" ([n, top], None for top = 0), "ws"}; nothing is copied to the host.
    Device-side problems (a bad row index or target) are read with blink_read_device_status(ws)."""
    rows, H = hidden.shape if getattr(hidden, "ndim", 0) == 2 else (None, None)
    _need("hidden", hidden, torch.bfloat16, (rows, H))
    V = unembed.shape[0] if getattr(unembed, "ndim", 0) == 2 else None
    _need("unembed", unembed, torch.bfloat16, (V, H), inner=2)
    n = rows
    if row_idx is not None:
        n = row_idx.numel()
        _need("row_idx", row_idx, torch.int32, (n,))
    if targets is not None:
        _need("targets", targets, torch.int32, (n,))
    if ws is not None:
        _need("ws", ws, torch.uint8, (ws.numel(),))
    _sizes(n, rows, V, H)
    top = _int32("top", int(top))
    with _Launch(stream, hidden, unembed, targets, row_idx, ws) as call:
        f32 = torch.float32
        logprob = None if targets is None else call.empty(f32, n)
        entropy, lse = call.empty(f32, n), call.empty(f32, n)
        ids, lps = (call.empty(torch.int32, n, top), call.empty(f32, n, top)) if top > 0 else (None, None)
        if ws is None:
            ws = call.workspace(token_logprobs_workspace_bytes(n, H, V, top))
        st = lib().blink_token_logprobs(
            hidden.data_ptr(), _row_stride(hidden) if rows else H, rows, _addr(row_idx), unembed.data_ptr(), V, H,
            _addr(targets), n, temperature, top, _addr(logprob), entropy.data_ptr(), lse.data_ptr(), _addr(ids), _addr(lps),
            ws.data_ptr(), ws.numel(), call.handle)
    _check(st, "blink_token_logprobs")
    return {"logprob": logprob, "entropy": entropy, "lse": lse, "top_ids": ids, "top_logprobs": lps, "ws": ws}


_E4M3, _E8M0, _BF16, _I32, _F32 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.bfloat16, torch.int32, torch.float32


def _usual_stream(stream, index):
    """The stream's handle where the call is on the current device and its current stream, else None.  The calls below
    check the usual arguments (contiguous, new outputs) in one expression each, which takes a fifth off a small call's
    time; whatever that expression does not let through takes the checks that say what is wrong, or that allow for
    strides, given outputs, other streams and devices."""
    if stream is None and index >= 0 and _raw_stream is not None and index == torch.cuda.current_device():
        return _raw_stream(index)
    return None


# ------------------------------------------------------------------------------------------------ rotary positions
ROPE_SCALINGS = {None: 0, "linear": 1, "base": 2, "by_dim": 3, "by_turns": 4}
_ROPE_TURNS = {"by_dim": (1.0, 32.0), "by_turns": (1.0, 4.0)}  # low and high where the caller gives none


def blink_rope_table(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0, original: int = 0,
                     low: float | None = None, high: float | None = None, device="cuda"):
    """Frequencies of the `rot` / 2 pairs that turn: (turns int64 [rot/2] on `device`, amplitude), to be kept for the
    calls that rotate.  `scaling`: None, "linear", "base", "by_dim" or "by_turns", for contexts `factor` times the
    `original` ones (include/blink.h has the formulas; `low` and `high` are turns over the original context)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALINGS)}, not {scaling!r}")
    rot = _int32("rot", rot)
    default = _ROPE_TURNS.get(scaling, (0.0, 0.0))
    turns = torch.empty(max(1, min(rot, 512) // 2), dtype=torch.int64)
    amplitude = ctypes.c_float(0.0)
    st = lib().blink_rope_table(rot, float(base), ROPE_SCALINGS[scaling], float(factor), _int32("original", original),
                                float(default[0] if low is None else low), float(default[1] if high is None else high),
                                turns.data_ptr(), ctypes.byref(amplitude))
    _check(st, "blink_rope_table")
    return turns.to(device), float(amplitude.value)


def _need_rows(name, t, n, H, d) -> int:
    """`t` is a bf16 CUDA tensor of shape (n, H, d) whose rows may be strided; returns their stride."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is torch.bfloat16 and t.shape == (n, H, d):
        row, head, one = t.stride()
        if one == 1 and head == d and n > 1:
            return row
    _refuse(name, t, torch.bfloat16, (n, H, d), 2)
    return t.stride(0) if n > 1 else H * d


def _turns_of(turns, d):
    n = turns.numel() if isinstance(turns, torch.Tensor) else None
    _need("turns", turns, torch.int64, (n,))
    if not 1 <= n <= d // 2:
        raise ValueError(f"turns must have 1..{d // 2} values (those of rot / 2 pairs), not {n}")
    return 2 * n


def blink_rope(q, k, positions, turns, interleaved: bool = False, amplitude: float = 1.0, q_out=None, k_out=None, stream=None):
    """Turn the heads of q [rows, Hq, d] and k [rows, Hkv, d] (None: q alone) bf16 by int32 `positions` [rows]: pairs
    (i, i + rot/2), or (2 i, 2 i + 1) if `interleaved`, with blink_rope_table's `turns` and amplitude.  Rows may be
    strided (slices of one projection).  q_out / k_out: None for new tensors, q / k themselves for in place.
    Returns (q_out, k_out)."""
    if k is not None and q_out is None and k_out is None:
        try:
            index = q.get_device()
            handle = _usual_stream(stream, index)
            (rows, Hq, d), Hkv, n = q.shape, k.shape[1], turns.shape[0]
            q_strides, k_strides = q.stride(), k.stride()
            if (handle is not None and q.dtype is _BF16 and k.dtype is _BF16 and positions.dtype is _I32 and turns.dtype is torch.int64 and
                    k.shape == (rows, Hkv, d) and positions.shape == (rows,) and turns.dim() == 1 and 1 <= n <= d // 2 and
                    k.get_device() == index and positions.get_device() == index and turns.get_device() == index and
                    q_strides[1] == d and q_strides[2] == 1 and k_strides[1] == d and k_strides[2] == 1 and 0 < rows <= INT32_MAX and
                    Hq <= INT32_MAX and Hkv <= INT32_MAX and positions.is_contiguous() and turns.is_contiguous()):
                q_out = torch.empty((rows, Hq, d), dtype=_BF16, device=q.device)
                k_out = torch.empty((rows, Hkv, d), dtype=_BF16, device=q.device)
        except (AttributeError, TypeError, ValueError, IndexError):
            pass
        if q_out is not None:
            one = rows == 1  # a single row has any stride
            st = lib().blink_rope(q.data_ptr(), Hq * d if one else q_strides[0], k.data_ptr(), Hkv * d if one else k_strides[0],
                                  positions.data_ptr(), rows, Hq, Hkv, d, 2 * n, turns.data_ptr(), amplitude, 1 if interleaved else 0,
                                  q_out.data_ptr(), Hq * d, k_out.data_ptr(), Hkv * d, handle)
            _check(st, "blink_rope")
            return q_out, k_out
    rows, Hq, d = q.shape if getattr(q, "ndim", 0) == 3 else (None,) * 3
    q_stride = _need_rows("q", q, rows, Hq, d)
    Hkv = k_stride = k_out_stride = 0
    if k is not None:
        Hkv = k.shape[1] if getattr(k, "ndim", 0) == 3 else None
        k_stride = _need_rows("k", k, rows, Hkv, d)
    elif k_out is not None:
        raise ValueError("k_out without k")
    _need("positions", positions, torch.int32, (rows,))
    rot = _turns_of(turns, d)
    _sizes(rows, Hq, Hkv, d)
    q_out_stride = Hq * d if q_out is None else _need_rows("q_out", q_out, rows, Hq, d)
    if k is not None:
        k_out_stride = Hkv * d if k_out is None else _need_rows("k_out", k_out, rows, Hkv, d)
    with _Launch(stream, q, k, positions, turns, q_out, k_out) as call:
        if q_out is None:
            q_out = call.empty(torch.bfloat16, rows, Hq, d)
        if k_out is None and k is not None:
            k_out = call.empty(torch.bfloat16, rows, Hkv, d)
        if rows:
            st = lib().blink_rope(q.data_ptr(), q_stride, _addr(k), k_stride, positions.data_ptr(), rows, Hq, Hkv, d, rot,
                                  turns.data_ptr(), amplitude, 1 if interleaved else 0, q_out.data_ptr(), q_out_stride, _addr(k_out),
                                  k_out_stride, call.handle)
            _check(st, "blink_rope")
    return q_out, k_out


# ------------------------------------------------------------------------------------------------ 8-bit paged cache
def blink_paged_cache(n_pages: int, page_tokens: int, Hkv: int, d: int, device="cuda") -> dict:
    """An empty cache of `n_pages` pages of `page_tokens` (16, 32, 64 or 128) tokens: {"k", "v": float8_e4m3fn
    [n_pages, Hkv, page_tokens, d], "k_scale", "v_scale": float8_e8m0fnu [n_pages, Hkv]}.  Any dict of such tensors is
    a cache: pages may be strided (K and V as halves of one tensor)."""
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=device)  # noqa: E731
    return {"k": zeros(n_pages, Hkv, page_tokens, d).view(torch.float8_e4m3fn),
            "v": zeros(n_pages, Hkv, page_tokens, d).view(torch.float8_e4m3fn),
            "k_scale": zeros(n_pages, Hkv).view(torch.float8_e8m0fnu), "v_scale": zeros(n_pages, Hkv).view(torch.float8_e8m0fnu)}


def _usual_cache(cache, table, index):
    """(sizes n, Hkv, page, d, arguments of the C calls, those of the table) of a contiguous cache and table on device
    `index`, else None."""
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    if not (k.dtype is _E4M3 and v.dtype is _E4M3 and ks.dtype is _E8M0 and vs.dtype is _E8M0 and table.dtype is _I32 and
            k.get_device() == index and v.get_device() == index and ks.get_device() == index and vs.get_device() == index and
            table.get_device() == index and k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and
            vs.is_contiguous() and table.is_contiguous()):
        return None
    shape, (S, width) = k.shape, table.shape
    n, Hkv, page, d = shape
    if not (v.shape == shape and ks.shape == (n, Hkv) and vs.shape == (n, Hkv) and 0 < n <= INT32_MAX and
            S <= INT32_MAX and width <= INT32_MAX):
        return None
    return (n, Hkv, page, d, (k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), Hkv * page * d, Hkv, n, page), S,
            (table.data_ptr(), width, width))


def _cache_of(cache, Hkv, d):
    """The tensors of a cache and its arguments of the C calls, checked."""
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    n, page = (k.shape[0], k.shape[2]) if getattr(k, "ndim", 0) == 4 else (None, None)
    _need("cache k", k, torch.float8_e4m3fn, (n, Hkv, page, d), inner=3)
    _need("cache k_scale", ks, torch.float8_e8m0fnu, (n, Hkv))
    strides, scale_strides = k.stride(), ks.stride()
    if not (isinstance(v, torch.Tensor) and v.is_cuda and v.dtype is torch.float8_e4m3fn and v.shape == k.shape and
            v.stride() == strides):
        _refuse("cache v", v, torch.float8_e4m3fn, (n, Hkv, page, d), 3)
    if not (isinstance(vs, torch.Tensor) and vs.is_cuda and vs.dtype is torch.float8_e8m0fnu and vs.shape == ks.shape and
            vs.stride() == scale_strides):
        _refuse("cache v_scale", vs, torch.float8_e8m0fnu, (n, Hkv), 1)
    if not 1 <= n <= INT32_MAX:
        raise ValueError(f"a cache has 1..{INT32_MAX} pages, not {n}")
    stride, scale_stride = strides[0], scale_strides[0]
    if n == 1:  # a single page has any stride
        stride, scale_stride = Hkv * page * d, Hkv
    elif v.stride(0) != stride or vs.stride(0) != scale_stride:
        raise ValueError("k and v of a cache, and their scales, must have the same page strides")
    return (k, v, ks, vs), (k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), stride, scale_stride, n, page)


def _table_of(table):
    rows, width = table.shape if getattr(table, "ndim", 0) == 2 else (None, None)
    _need("page_table", table, torch.int32, (rows, width))
    if width > INT32_MAX or rows > INT32_MAX:
        _sizes(rows, width)
    return rows, (table.data_ptr(), table.stride(0) if rows > 1 else width, width)


def _bytes(name, ws):
    if ws is not None:
        _need(name, ws, torch.uint8, (ws.numel(),))


def paged_append_workspace_bytes() -> int:
    return int(lib().blink_paged_append_workspace())


def blink_paged_append(k, v, cache: dict, page_table, cu_new, start, max_new: int, positions=None, turns=None,
                       interleaved: bool = False, amplitude: float = 1.0, ws=None, stream=None):
    """Write the new tokens k, v [n, Hkv, d] bf16 (rows may be strided) of S sequences into their pages: sequence s's
    rows [cu_new[s], cu_new[s+1]) follow its start[s] tokens; page_table [S, width], cu_new [S+1], start [S] int32.
    Keys are turned by `positions` (int32 [n]; None: start + 0, 1, ...) with blink_rope_table's `turns` and amplitude
    (turns None: they are rotated already).  max_new: upper bound of a sequence's new tokens.  Returns ws; device-side
    problems (a bad length or page) are read with blink_read_device_status(ws)."""
    max_new = _int32("max_new", max_new)
    try:
        index = k.get_device()
        handle = _usual_stream(stream, index)
        usual = None if handle is None else _usual_cache(cache, page_table, index)
        if usual is not None:
            n, Hkv, d = k.shape
            _, heads, _, width, args, S, table = usual
            if not (v.shape == k.shape and heads == Hkv and width == d and k.dtype is _BF16 and v.dtype is _BF16 and
                    v.get_device() == index and 0 < n <= INT32_MAX and k.stride()[1:] == (d, 1) and v.stride()[1:] == (d, 1) and
                    cu_new.dtype is _I32 and start.dtype is _I32 and cu_new.shape == (S + 1,) and start.shape == (S,) and
                    cu_new.get_device() == index and start.get_device() == index and cu_new.is_contiguous() and
                    start.is_contiguous() and positions is None and
                    (turns is None or (turns.dtype is torch.int64 and turns.get_device() == index and turns.dim() == 1 and
                                       turns.is_contiguous() and 1 <= turns.shape[0] <= d // 2)) and
                    (ws is None or (ws.dtype is torch.uint8 and ws.get_device() == index and ws.is_contiguous()))):
                usual = None
    except (AttributeError, TypeError, ValueError):
        usual = None
    if usual is not None:
        if ws is None:
            ws = _Launch(None, k).workspace(paged_append_workspace_bytes())
        row = Hkv * d  # a single row has any stride
        st = lib().blink_paged_append(k.data_ptr(), k.stride(0) if n > 1 else row, v.data_ptr(), v.stride(0) if n > 1 else row,
                                      n, Hkv, d, *args, *table,
                                      cu_new.data_ptr(), start.data_ptr(), S, max_new, None, _addr(turns),
                                      0 if turns is None else 2 * turns.shape[0], amplitude, 1 if interleaved else 0,
                                      ws.data_ptr(), ws.numel(), handle)
        _check(st, "blink_paged_append")
        return ws
    n, Hkv, d = k.shape if getattr(k, "ndim", 0) == 3 else (None,) * 3
    k_stride, v_stride = _need_rows("k", k, n, Hkv, d), _need_rows("v", v, n, Hkv, d)
    tensors, args = _cache_of(cache, Hkv, d)
    S, table = _table_of(page_table)
    _need("cu_new", cu_new, torch.int32, (S + 1,))
    _need("start", start, torch.int32, (S,))
    if positions is not None:
        _need("positions", positions, torch.int32, (n,))
    rot = 0 if turns is None else _turns_of(turns, d)
    _bytes("ws", ws)
    _sizes(n, S)
    with _Launch(stream, k, v, *tensors, page_table, cu_new, start, positions, turns, ws) as call:
        if ws is None:
            ws = call.workspace(paged_append_workspace_bytes())
        if n:
            st = lib().blink_paged_append(k.data_ptr(), k_stride, v.data_ptr(), v_stride, n, Hkv, d, *args, *table,
                                          cu_new.data_ptr(), start.data_ptr(), S, max_new, _addr(positions), _addr(turns), rot,
                                          amplitude, 1 if interleaved else 0, ws.data_ptr(), ws.numel(), call.handle)
            _check(st, "blink_paged_append")
    return ws


def paged_token_attention_workspace_bytes(S, T, max_len, Hq, Hkv, d) -> int:
    return int(lib().blink_paged_token_attention_workspace(int(S), int(T), int(max_len), int(Hq), int(Hkv), int(d)))


def blink_paged_token_attention(q, cache: dict, page_table, length, max_len: int, scale: float = 0.0, out=None, lse=None,
                                want_lse: bool = False, ws=None, stream=None):
    """Attention of the last T tokens of S sequences, q [S, T, Hq, d] bf16, over the pages that hold them: sequence s
    has length[s] (int32, on the device) tokens in row s of page_table, and token t sees the first length - T + 1 + t.
    max_len: upper bound of `length`.  Returns (out [S, T, Hq, d], lse [Hq, S * T] or None, ws)."""
    max_len = _int32("max_len", max_len)
    try:
        index = q.get_device()
        handle = _usual_stream(stream, index)
        usual = None if handle is None else _usual_cache(cache, page_table, index)
        if usual is not None:
            S, T, Hq, d = q.shape
            _, Hkv, _, width, args, rows, table = usual
            if not (width == d and rows == S and q.dtype is _BF16 and q.is_contiguous() and length.dtype is _I32 and
                    length.shape == (S,) and length.get_device() == index and length.is_contiguous() and
                    T <= INT32_MAX and Hq <= INT32_MAX and out is None and lse is None and
                    (ws is None or (ws.dtype is torch.uint8 and ws.get_device() == index and ws.is_contiguous()))):
                usual = None
    except (AttributeError, TypeError, ValueError):
        usual = None
    if usual is not None:
        out = torch.empty_like(q)
        lse = torch.empty((Hq, S * T), dtype=_F32, device=q.device) if want_lse else None
        if ws is None:
            ws = _Launch(None, q).workspace(paged_token_attention_workspace_bytes(S, T, max_len, Hq, Hkv, d))
        st = lib().blink_paged_token_attention(q.data_ptr(), *args, *table, length.data_ptr(), S, T, max_len, Hq, Hkv, d, scale,
                                               out.data_ptr(), _addr(lse), ws.data_ptr(), ws.numel(), handle)
        _check(st, "blink_paged_token_attention")
        return out, lse, ws
    S, T, Hq, d = q.shape if getattr(q, "ndim", 0) == 4 else (None,) * 4
    _need("q", q, torch.bfloat16, (S, T, Hq, d), inner=4)
    Hkv = cache["k"].shape[1] if getattr(cache["k"], "ndim", 0) == 4 else None
    tensors, args = _cache_of(cache, Hkv, d)
    rows, table = _table_of(page_table)
    _sizes(T, Hq)
    if rows != S:
        raise ValueError(f"page_table must have a row for each of {S} sequences, not {rows}")
    _need("length", length, torch.int32, (S,))
    if out is not None:
        _need("out", out, torch.bfloat16, (S, T, Hq, d), inner=4)
    if lse is not None:
        _need("lse", lse, torch.float32, (Hq, S * T), inner=2)
    _bytes("ws", ws)
    with _Launch(stream, q, *tensors, page_table, length, out, lse, ws) as call:
        if out is None:
            out = torch.empty_like(q)
        if lse is None and want_lse:
            lse = call.empty(torch.float32, Hq, S * T)
        if ws is None:
            ws = call.workspace(paged_token_attention_workspace_bytes(S, T, max_len, Hq, Hkv, d))
        st = lib().blink_paged_token_attention(q.data_ptr(), *args, *table, length.data_ptr(), S, T, max_len, Hq, Hkv, d, scale,
                                               out.data_ptr(), _addr(lse), ws.data_ptr(), ws.numel(), call.handle)
    _check(st, "blink_paged_token_attention")
    return out, lse, ws


def _int32s(name, values):
    """A host list as an array of int32 (and its address)."""
    try:
        a = array.array("i", values)
    except OverflowError:
        raise ValueError(f"{name} must fit 32 bits: {list(values)}") from None
    return a, a.buffer_info()[0]


def paged_prefix_tail_workspace_bytes(req_rows, prefix_len, B, Hq, Hkv, d) -> int:
    if len(req_rows) != len(prefix_len) + 1:
        raise ValueError("req_rows must have one value more than prefix_len")
    rows, at_rows = _int32s("req_rows", req_rows)
    lens, at_lens = _int32s("prefix_len", prefix_len)
    return int(lib().blink_paged_prefix_tail_workspace(at_rows, at_lens, len(lens), int(B), int(Hq), int(Hkv), int(d)))


def blink_paged_prefix_tail_attention(q, cache: dict, page_table, prefix_len, k_tail, v_tail, cu_seqlens, B: int, max_tail: int,
                                      req_rows=None, seq_start=None, scale: float = 0.0, out=None, lse=None,
                                      want_lse: bool = False, ws=None, stream=None):
    """Prefix-tail attention with the prefixes in pages: request r owns rows [req_rows[r], req_rows[r+1]) of q
    [rows, Hq, d] and k_tail / v_tail [rows, Hkv, d] bf16 (req_rows None: one request has them all) and attends to the
    first prefix_len[r] tokens of row r of page_table.  prefix_len and req_rows are host lists; the rest as
    blink_prefix_tail_attention.  Returns (out, lse, ws)."""
    B, max_tail = _int32("B", B), _int32("max_tail", max_tail)
    try:
        index = q.get_device()
        handle = _usual_stream(stream, index)
        usual = None if handle is None else _usual_cache(cache, page_table, index)
        if usual is not None:
            rows, Hq, d = q.shape
            _, Hkv, _, width, args, n_req, table = usual
            if not (width == d and q.dtype is _BF16 and k_tail.dtype is _BF16 and v_tail.dtype is _BF16 and
                    cu_seqlens.dtype is _I32 and k_tail.shape == (rows, Hkv, d) and v_tail.shape == (rows, Hkv, d) and
                    cu_seqlens.shape == (B + 1,) and k_tail.get_device() == index and v_tail.get_device() == index and
                    cu_seqlens.get_device() == index and q.is_contiguous() and k_tail.is_contiguous() and v_tail.is_contiguous() and
                    cu_seqlens.is_contiguous() and seq_start is None and out is None and lse is None and rows <= INT32_MAX and
                    Hq <= INT32_MAX and (ws is None or (ws.dtype is torch.uint8 and ws.get_device() == index and ws.is_contiguous()))):
                usual = None
    except (AttributeError, TypeError, ValueError):
        usual = None
    if usual is None:
        rows, Hq, d = q.shape if getattr(q, "ndim", 0) == 3 else (None,) * 3
        _need("q", q, torch.bfloat16, (rows, Hq, d), inner=3)
        Hkv = k_tail.shape[1] if getattr(k_tail, "ndim", 0) == 3 else None
        _need("k_tail", k_tail, torch.bfloat16, (rows, Hkv, d), inner=3)
        _need("v_tail", v_tail, torch.bfloat16, (rows, Hkv, d), inner=3)
        tensors, args = _cache_of(cache, Hkv, d)
        n_req, table = _table_of(page_table)
        _need("cu_seqlens", cu_seqlens, torch.int32, (B + 1,))
        if seq_start is not None:
            _need("seq_start", seq_start, torch.int32, (B,))
        if out is not None:
            _need("out", out, torch.bfloat16, (rows, Hq, d), inner=3)
        if lse is not None:
            _need("lse", lse, torch.float32, (Hq, rows), inner=2)
        _bytes("ws", ws)
        _sizes(rows, Hq, n_req)
    if req_rows is None:
        req_rows = [0, rows]
    if len(prefix_len) != n_req or len(req_rows) != n_req + 1:
        raise ValueError(f"page_table has {n_req} requests: prefix_len needs as many values, req_rows one more")
    (host_rows, h_rows), (host_len, h_len) = _int32s("req_rows", req_rows), _int32s("prefix_len", prefix_len)  # read by the call
    if usual is not None:
        out = torch.empty_like(q)
        lse = torch.empty((Hq, rows), dtype=_F32, device=q.device) if want_lse else None
        if ws is None:
            ws = _Launch(None, q).workspace(paged_prefix_tail_workspace_bytes(req_rows, prefix_len, B, Hq, Hkv, d))
        st = lib().blink_paged_prefix_tail_attention(
            q.data_ptr(), *args, *table, k_tail.data_ptr(), v_tail.data_ptr(), cu_seqlens.data_ptr(), None, B, rows, n_req, h_rows,
            h_len, max_tail, Hq, Hkv, d, scale, out.data_ptr(), _addr(lse), ws.data_ptr(), ws.numel(), handle)
        _check(st, "blink_paged_prefix_tail_attention")
        return out, lse, ws
    with _Launch(stream, q, *tensors, page_table, k_tail, v_tail, cu_seqlens, seq_start, out, lse, ws) as call:
        if out is None:
            out = torch.empty_like(q)
        if lse is None and want_lse:
            lse = call.empty(torch.float32, Hq, rows)
        if ws is None:
            ws = call.workspace(paged_prefix_tail_workspace_bytes(req_rows, prefix_len, B, Hq, Hkv, d))
        st = lib().blink_paged_prefix_tail_attention(
            q.data_ptr(), *args, *table, k_tail.data_ptr(), v_tail.data_ptr(), cu_seqlens.data_ptr(), _addr(seq_start), B, rows,
            n_req, h_rows, h_len, max_tail, Hq, Hkv, d, scale, out.data_ptr(), _addr(lse), ws.data_ptr(), ws.numel(), call.handle)
    _check(st, "blink_paged_prefix_tail_attention")
    return out, lse, ws
