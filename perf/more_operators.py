"""Measured calls of the 8-bit paged cache: rotary positions, appending, and the attention over its pages.

Four operators: the rotation of queries and keys by their positions (``rope``), keys and values written into
the pages of an 8-bit cache with the rotation on the way (``append``), attention of each sequence's last tokens
over its pages (``token``), and the attention of question tails over a shared prefix held in pages (``tail``).
``run`` computes them with elementary torch operations in 32 bits (angles in 64), or, where ``own`` is true,
through the library.

A page holds ``page`` tokens of every kv head: codes in e4m3 and, per kv head, one power of two for K and one for
V.  With m the largest magnitude among the page's tokens the scale is the smallest 2^e with m <= 448 * 2^e, e kept
in -48..32; it never shrinks while a page fills, and when it grows the codes that were there are rounded again.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
E_MIN, E_MAX = -48, 32  # exponents of the pages' scales


# ------------------------------------------------------------------------------------------ cases
def _rope(name, rows, Hq, Hkv, d, rot, interleaved, scaling, far):
    return {"name": name, "op": "rope", "rows": rows, "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rot, "interleaved": interleaved,
            "scaling": scaling, "far": far}


def _append(name, S, new, start, Hkv, d, page, rot, interleaved):
    return {"name": name, "op": "append", "S": S, "new": new, "start": start, "Hkv": Hkv, "d": d, "page": page, "rot": rot,
            "interleaved": interleaved}


def _token(name, S, T, longest, Hq, Hkv, d, page):
    return {"name": name, "op": "token", "S": S, "T": T, "longest": longest, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page}


def _tail(name, requests, P, questions, shortest, longest, Hq, Hkv, d, page):
    return {"name": name, "op": "tail", "requests": requests, "P": P, "questions": questions, "shortest": shortest,
            "longest": longest, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page}


def listed():
    return [
        # the next token of 64 sequences somewhere in a long context: latency
        _rope("rope_token", 64, 32, 8, 128, 128, False, "by_turns", 131072),
        # the tails of the 2k workload, half of each head rotated in the interleaved layout
        _rope("rope_2k", 1275, 32, 8, 128, 64, True, "none", 2048 + 128),
        # the whole long document, positions stretched over a long context
        _rope("rope_18k", 18432, 32, 8, 128, 128, False, "by_dim", 18432),
        # one new token for each of 64 sequences, in pages that are partly full
        _append("append_token", 64, 1, 18000, 8, 128, 64, 128, False),
        # pieces of prompts of several users, each continuing in the middle of a small page
        _append("append_pieces", 16, 511, 1000, 5, 64, 16, 32, True),
        # the whole long document into empty pages
        _append("append_18k", 1, 18432, 0, 8, 128, 64, 128, False),
        # a small model's next token for four sequences: launch latency
        _token("token_tiny", 4, 1, 64, 4, 2, 64, 16),
        # one token of one sequence against the long document
        _token("token_one", 1, 1, 18432, 32, 8, 128, 64),
        # the next token of 64 sequences of many lengths
        _token("token_batch", 64, 1, 18432, 32, 8, 128, 64),
        # the tiny workload: four questions against a 64-token prompt
        _tail("tail_tiny", 1, 64, 4, 8, 24, 4, 2, 64, 16),
        # sixteen questions against a 2k prompt
        _tail("tail_2k", 1, 2048, 16, 32, 128, 32, 8, 128, 64),
        # the long-document workload: 64 questions against 18432 tokens
        _tail("tail_18k", 1, 18432, 64, 64, 256, 32, 8, 128, 64),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(4, 2, 64), (32, 8, 128), (40, 8, 128), (8, 8, 64), (16, 2, 128), (5, 1, 64), (28, 4, 128)]


def draw(rng):
    op = rng.choice(["rope", "append", "token", "tail"])
    Hq, Hkv, d = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
        rows = _log_uniform(rng, 1, 18432 * 40 * 128 // ((Hq + Hkv) * d) // 2)
        scaling = rng.choice(["none", "linear", "base", "by_dim", "by_turns"])
        c = _rope("", rows, Hq, Hkv, d, rot, rng.random() < 0.5, scaling if rot > 2 else "none", _log_uniform(rng, 1, 131072))
    elif op == "append":
        S = _log_uniform(rng, 1, 64)
        new = _log_uniform(rng, 1, max(1, min(120000, 18432 * 1024 // (S * Hkv * d))))
        c = _append("", S, new, rng.choice([0, rng.randint(1, 4000)]), Hkv, d, page, rng.choice([d, d // 2, 2 * rng.randint(1, d // 2)]),
                    rng.random() < 0.5)
    elif op == "token":
        S = _log_uniform(rng, 1, 64)
        T = rng.choice([1, 1, 1, 2, 4])
        c = _token("", S, T, T + _log_uniform(rng, 1, min(131000, 18432 * 64 * 1024 // (S * Hkv * d) - T)), Hq, Hkv, d, page)
    else:
        requests = rng.choice([1, 1, 1, 2, 4])
        P = _log_uniform(rng, 1, 18432 * 32 // max(32, Hq) // requests)
        questions = _log_uniform(rng, 1, 64 // requests)
        shortest = _log_uniform(rng, 1, 64)
        c = _tail("", requests, P, questions, shortest, shortest + rng.randint(0, 192), Hq, Hkv, d, page)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------ sizes
def _sizes_of(c):
    """What is ragged in a case: the same sizes for every seed."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    if c["op"] == "append":  # every sequence's new tokens and the length it has
        new = [c["new"] if c["S"] == 1 or c["new"] == 1 else r.randint(1, c["new"]) for _ in range(c["S"])]
        start = [r.randint(c["start"] // 2, c["start"]) for _ in range(c["S"])]
        return new, start
    if c["op"] == "token":  # every sequence's length, its last T tokens included
        return [c["longest"]] + [r.randint(c["T"], c["longest"]) for _ in range(c["S"] - 1)]
    if c["op"] == "tail":  # the requests' prefixes, and their questions' tails
        prefix = [c["P"]] + [r.randint(1, c["P"]) for _ in range(c["requests"] - 1)]
        tails = [[r.randint(c["shortest"], c["longest"]) for _ in range(c["questions"])] for _ in range(c["requests"])]
        return prefix, tails
    return None


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------------------------------------ inputs
BASE, FACTOR, ORIGINAL = 500000.0, 8.0, 8192
SCALINGS = {"none": {}, "linear": {"factor": FACTOR}, "base": {"factor": FACTOR},
            "by_dim": {"factor": FACTOR, "original": ORIGINAL, "low": 1.0, "high": 32.0},
            "by_turns": {"factor": FACTOR, "original": ORIGINAL, "low": 1.0, "high": 4.0}}


def _frequencies(rot, scaling):
    """Radians per position of each pair, and the factor of the rotated values."""
    n = rot // 2
    base = BASE * FACTOR ** (rot / (rot - 2)) if scaling == "base" else BASE
    f = [base ** (-2.0 * i / rot) for i in range(n)]
    if scaling == "linear":
        return [x / FACTOR for x in f], 1.0
    if scaling == "by_dim":  # pairs below `lo` keep their frequency, those from `hi` on are stretched
        where = lambda turns: rot * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(BASE))  # noqa: E731
        lo, hi = max(0, math.floor(where(32.0))), min(rot - 1, math.ceil(where(1.0)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(n)]
        return [x * (1 - r + r / FACTOR) for x, r in zip(f, ramp)], 0.1 * math.log(FACTOR) + 1.0
    if scaling == "by_turns":  # pairs that turn often over the original context keep their frequency
        share = [min(1.0, max(0.0, (ORIGINAL * x / (2 * math.pi) - 1.0) / (4.0 - 1.0))) for x in f]
        return [x * (s + (1 - s) / FACTOR) for x, s in zip(f, share)], 1.0
    return f, 1.0


def _table(st, rot, scaling):
    """The frequencies that a program keeps: the library's table, or the plain ones."""
    if own:
        from shared_prefix_question_gb300 import blink
        st["turns"], st["amplitude"] = blink.blink_rope_table(rot, BASE, scaling=None if scaling == "none" else scaling, device=DEV,
                                                              **SCALINGS[scaling])
    else:
        f, st["amplitude"] = _frequencies(rot, scaling)
        st["freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _prepare_rope(c, seed):
    g = _gen(seed)
    rows, Hq, Hkv, d = c["rows"], c["Hq"], c["Hkv"], c["d"]
    # q and k as the projection leaves them: slices of one row
    qkv = torch.randn(rows, (Hq + 2 * Hkv) * d, device=DEV, generator=g).to(torch.bfloat16)
    st = {"q": qkv[:, :Hq * d].view(rows, Hq, d), "k": qkv[:, Hq * d:(Hq + Hkv) * d].view(rows, Hkv, d)}
    if rows == c["far"]:  # a whole document
        st["pos"] = torch.arange(rows, dtype=torch.int32, device=DEV)
    else:
        st["pos"] = torch.randint(0, c["far"], (rows,), device=DEV, generator=g).to(torch.int32)
    _table(st, c["rot"], c["scaling"])
    return st


def _prepare_append(c, seed):
    g = _gen(seed)
    S, Hkv, d, page = c["S"], c["Hkv"], c["d"], c["page"]
    new, start = _sizes_of(c)
    n = sum(new)
    need = [_pages(a + b, page) for a, b in zip(start, new)]
    total, widest = sum(need) + 3, max(need)
    perm = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    table = torch.full((S, widest), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s in range(S):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
    # keys have a few wide channels, tokens differ in size; what the pages hold already is a little smaller on average
    wide = torch.exp(0.7 * torch.randn(Hkv, d, device=DEV, generator=g))
    k = (torch.randn(n, Hkv, d, device=DEV, generator=g) * wide * torch.exp(0.3 * torch.randn(n, 1, 1, device=DEV, generator=g)))
    v = torch.randn(n, Hkv, d, device=DEV, generator=g) * torch.exp(0.5 * torch.randn(n, Hkv, 1, device=DEV, generator=g))
    st = {"k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16), "table": table,
          "cu": torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32, device=DEV),
          "start": torch.tensor(start, dtype=torch.int32, device=DEV), "max_new": max(new)}
    cache = {}
    for name in ("k", "v"):
        codes = torch.zeros(total, Hkv, page, d, dtype=torch.uint8, device=DEV)
        scale = torch.zeros(total, Hkv, dtype=torch.uint8, device=DEV)
        if max(start) > 0:
            codes.copy_((100.0 * torch.randn(total, Hkv, page, d, device=DEV, generator=g)).clamp(-448, 448)
                        .to(torch.float8_e4m3fn).view(torch.uint8))
            scale.copy_(127 + torch.randint(-8, -5, (total, Hkv), device=DEV, generator=g).to(torch.uint8))
        cache[name], cache[name + "_scale"] = codes.view(torch.float8_e4m3fn), scale.view(torch.float8_e8m0fnu)
    st["cache"] = cache
    _table(st, c["rot"], "none")
    if own:
        from shared_prefix_question_gb300 import blink
        st["ws"] = blink.new_workspace(blink.paged_append_workspace_bytes(), DEV)
    return st


def _filled_cache(g, tokens, Hkv, d, page):
    """Pages that hold sequences of `tokens` tokens in any order, and the table of the pages."""
    need = [_pages(t, page) for t in tokens]
    total = sum(need) + 2
    perm = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    table = torch.full((len(tokens), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = perm[at:at + m]
        at += m
    cache = {}
    for name in ("k", "v"):
        # codes of normal values: the largest of a page near 448, the scale about one hundredth
        size = 110.0 * torch.exp(0.2 * torch.randn(total, Hkv, page, 1, device=DEV, generator=g))
        x = torch.empty(total, Hkv, page, d, dtype=torch.float8_e4m3fn, device=DEV)
        for a in range(0, total, 1024):
            b = min(total, a + 1024)
            x[a:b] = (torch.randn(b - a, Hkv, page, d, device=DEV, generator=g) * size[a:b]).clamp(-448, 448).to(torch.float8_e4m3fn)
        cache[name] = x
        cache[name + "_scale"] = (127 + torch.randint(-8, -5, (total, Hkv), device=DEV, generator=g)).to(torch.uint8).view(
            torch.float8_e8m0fnu)
    return cache, table


def _prepare_token(c, seed):
    g = _gen(seed)
    lens = _sizes_of(c)
    cache, table = _filled_cache(g, lens, c["Hkv"], c["d"], c["page"])
    q = torch.randn(c["S"], c["T"], c["Hq"], c["d"], device=DEV, generator=g).to(torch.bfloat16)
    st = {"cache": cache, "table": table, "q": q, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    if own:
        from shared_prefix_question_gb300 import blink
        st["ws"] = blink.new_workspace(
            blink.paged_token_attention_workspace_bytes(c["S"], c["T"], c["longest"], c["Hq"], c["Hkv"], c["d"]), DEV)
    return st


def _prepare_tail(c, seed):
    g = _gen(seed)
    prefix, tails = _sizes_of(c)
    cache, table = _filled_cache(g, prefix, c["Hkv"], c["d"], c["page"])
    flat = [t for r in tails for t in r]
    rows = sum(flat)
    bf = lambda H: torch.randn(rows, H, c["d"], device=DEV, generator=g).to(torch.bfloat16)  # noqa: E731
    st = {"cache": cache, "table": table, "q": bf(c["Hq"]), "k": bf(c["Hkv"]), "v": bf(c["Hkv"]),
          "cu": torch.tensor([sum(flat[:i]) for i in range(len(flat) + 1)], dtype=torch.int32, device=DEV),
          "prefix": prefix, "req_rows": [sum(sum(r) for r in tails[:i]) for i in range(len(tails) + 1)], "max_tail": max(flat),
          "B": len(flat)}
    st["prefix_dev"], st["req_rows_dev"] = (torch.tensor(x, device=DEV) for x in (prefix, st["req_rows"]))
    if own:
        from shared_prefix_question_gb300 import blink
        st["ws"] = blink.new_workspace(
            blink.paged_prefix_tail_workspace_bytes(st["req_rows"], prefix, st["B"], c["Hq"], c["Hkv"], c["d"]), DEV)
    return st


def prepare(case, seed):
    st = {"rope": _prepare_rope, "append": _prepare_append, "token": _prepare_token, "tail": _prepare_tail}[case["op"]](case, seed)
    st["case"] = case
    return st


# ------------------------------------------------------------------------------------------ passes
def _rotated(x, pos, st, rot, interleaved):
    """x [n, H, d] in 32 bits, its first `rot` values of each head turned by their positions."""
    angle = pos.double().unsqueeze(1) * st["freq"]
    cos = (angle.cos() * st["amplitude"]).float().unsqueeze(1)
    sin = (angle.sin() * st["amplitude"]).float().unsqueeze(1)
    out = x.float()
    a, b = (out[..., 0:rot:2], out[..., 1:rot:2]) if interleaved else (out[..., :rot // 2], out[..., rot // 2:rot])
    c, s = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([c, s], dim=-1).flatten(-2) if interleaved else torch.cat([c, s], dim=-1)
    return torch.cat([turned, out[..., rot:]], dim=-1)


def _run_rope(st):
    c = st["case"]
    if own:
        from shared_prefix_question_gb300 import blink
        q, k = blink.blink_rope(st["q"], st["k"], st["pos"], st["turns"], interleaved=c["interleaved"], amplitude=st["amplitude"])
        return {"q": q, "k": k}
    return {"q": _rotated(st["q"], st["pos"], st, c["rot"], c["interleaved"]).to(torch.bfloat16),
            "k": _rotated(st["k"], st["pos"], st, c["rot"], c["interleaved"]).to(torch.bfloat16)}


def _write(x, codes, scale, page_of, slot, first, filled, page):
    """x [n, Hkv, d] (32 bits) into slot `slot` of page `page_of`; page first[s] holds filled[s] tokens already."""
    total, Hkv = scale.shape
    old = scale.view(torch.uint8).to(torch.int32) - 127
    most = torch.zeros(total, Hkv, device=x.device).index_reduce_(0, page_of, x.abs().amax(dim=-1), "amax")
    m, e = torch.frexp(most)
    e = torch.where(most > 0, torch.where(m <= 0.875, e - 9, e - 8), torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    touched = torch.zeros(total, dtype=torch.bool, device=x.device).index_fill_(0, page_of, True)
    keeps = torch.zeros(total, dtype=torch.int64, device=x.device).index_put_((first,), filled)  # tokens there before
    e = torch.where((keeps > 0).unsqueeze(1), torch.maximum(e, old), e)
    e = torch.where(touched.unsqueeze(1), e, old)
    # what was in a page whose scale grew is rounded again
    there = codes.view(torch.uint8)[first].view(torch.float8_e4m3fn).float() * torch.exp2((old - e)[first].float())[:, :, None, None]
    mine = (torch.arange(page, device=x.device) < filled.unsqueeze(1))[:, None, :, None]
    again = torch.where(mine, there.to(torch.float8_e4m3fn).view(torch.uint8), codes.view(torch.uint8)[first])
    codes.view(torch.uint8).index_put_((first,), again)
    new = (x * torch.exp2(-e[page_of].float()).unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    codes.view(torch.uint8).permute(0, 2, 1, 3).index_put_((page_of, slot), new.view(torch.uint8))
    scale.view(torch.uint8).copy_((e + 127).to(torch.uint8))


def _run_append(st):
    c, cache = st["case"], st["cache"]
    if own:
        from shared_prefix_question_gb300 import blink
        blink.blink_paged_append(st["k"], st["v"], cache, st["table"], st["cu"], st["start"], st["max_new"], turns=st["turns"],
                                 interleaved=c["interleaved"], amplitude=st["amplitude"], ws=st["ws"])
        return cache
    n, page = st["k"].shape[0], c["page"]
    cu, start = st["cu"].long(), st["start"].long()
    token = torch.arange(n, device=cu.device)
    seq = torch.searchsorted(cu, token, right=True) - 1
    pos = start[seq] + token - cu[seq]
    page_of = st["table"][seq, pos // page].long()
    slot = pos % page
    first = torch.gather(st["table"], 1, (start // page).unsqueeze(1)).squeeze(1).long()
    _write(_rotated(st["k"], pos, st, c["rot"], c["interleaved"]), cache["k"], cache["k_scale"], page_of, slot, first, start % page, page)
    _write(st["v"].float(), cache["v"], cache["v_scale"], page_of, slot, first, start % page, page)
    return cache


def _values(cache, name, table):
    """[S, Hkv, pages * page, d] in 32 bits: what the pages of `table` stand for (those of -1 are not used)."""
    at = table.clamp(min=0).long()
    x = cache[name].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    x = x * torch.exp2(cache[name + "_scale"].view(torch.uint8)[at].float() - 127.0)[..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _run_token(st):
    c = st["case"]
    S, T, Hq, Hkv, d = c["S"], c["T"], c["Hq"], c["Hkv"], c["d"]
    if own:
        from shared_prefix_question_gb300 import blink
        out, lse, _ = blink.blink_paged_token_attention(st["q"], st["cache"], st["table"], st["lens"], c["longest"], want_lse=True,
                                                        ws=st["ws"])
        return {"out": out, "lse": lse}
    g = Hq // Hkv
    q = st["q"].float().view(S, T, Hkv, g, d).permute(0, 2, 1, 3, 4).reshape(S, Hkv, T * g, d)
    s = torch.matmul(q, _values(st["cache"], "k", st["table"]).transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    see = st["lens"].unsqueeze(1) - (T - 1 - torch.arange(T, device=s.device))  # [S, T] keys that each token sees
    hidden = torch.arange(s.shape[-1], device=s.device) >= see.repeat_interleave(g, dim=1).unsqueeze(-1)
    s.masked_fill_(hidden.unsqueeze(1), -math.inf)
    most = s.amax(dim=-1, keepdim=True)
    p = s.sub_(most).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, _values(st["cache"], "v", st["table"])) / total
    lse = (most + total.log()).squeeze(-1).view(S, Hkv, T, g).permute(1, 3, 0, 2).reshape(Hq, S * T)
    return {"out": o.view(S, Hkv, T, g, d).permute(0, 2, 1, 3, 4).reshape(S, T, Hq, d).to(torch.bfloat16), "lse": lse}


def _run_tail(st):
    c = st["case"]
    rows, Hq, d = st["q"].shape
    Hkv = c["Hkv"]
    if own:
        from shared_prefix_question_gb300 import blink
        out, lse, _ = blink.blink_paged_prefix_tail_attention(
            st["q"], st["cache"], st["table"], st["prefix"], st["k"], st["v"], st["cu"], st["B"], st["max_tail"],
            req_rows=st["req_rows"], want_lse=True, ws=st["ws"])
        return {"out": out, "lse": lse}
    g, R = Hq // Hkv, len(st["prefix"])
    row = torch.arange(rows, device=DEV)
    req = torch.searchsorted(st["req_rows_dev"], row, right=True) - 1
    cu = st["cu"].long()
    begin = cu[torch.searchsorted(cu, row, right=True) - 1]
    k, v = (_values(st["cache"], x, st["table"]).transpose(0, 1).flatten(1, 2) for x in ("k", "v"))  # [Hkv, R * L, d]
    L = k.shape[1] // R
    key = torch.arange(L, device=DEV)
    mine = (torch.arange(R, device=DEV).unsqueeze(1) == req[:, None, None]) & (key < st["prefix_dev"].unsqueeze(1))
    see = torch.cat([mine.flatten(1), (row >= begin.unsqueeze(1)) & (row <= row.unsqueeze(1))], dim=1)  # [rows, keys]
    k = torch.cat([k, st["k"].float().transpose(0, 1)], dim=1)
    v = torch.cat([v, st["v"].float().transpose(0, 1)], dim=1)
    q = st["q"].float().view(rows, Hkv, g, d).permute(1, 2, 0, 3).reshape(Hkv, g * rows, d)
    s = torch.bmm(q, k.transpose(1, 2)).mul_(1.0 / math.sqrt(d))
    s.view(Hkv, g, rows, -1).masked_fill_(~see, -math.inf)
    most = s.amax(dim=-1, keepdim=True)
    p = s.sub_(most).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.bmm(p, v).div_(total)
    return {"out": o.view(Hkv, g, rows, d).permute(2, 0, 1, 3).reshape(rows, Hq, d).to(torch.bfloat16),
            "lse": (most + total.log()).view(Hq, rows)}


def run(state):
    return {"rope": _run_rope, "append": _run_append, "token": _run_token, "tail": _run_tail}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "rope":  # every row read and written once
        values = c["rows"] * (c["Hq"] + c["Hkv"]) * c["d"]
        return {"bytes": 4 * values + 4 * c["rows"] + 8 * (c["rot"] // 2), "flops": 3 * c["rows"] * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "append":  # 16-bit rows read, 8-bit rows written, the scales of the pages they fall into
        new, start = _sizes_of(c)
        n = sum(new)
        pages = sum(_pages(a + b, c["page"]) - a // c["page"] for a, b in zip(start, new))
        return {"bytes": n * c["Hkv"] * c["d"] * 2 * 3 + pages * (4 + 4 * c["Hkv"]), "flops": 3 * n * c["Hkv"] * c["rot"]}
    if c["op"] == "token":  # codes and scales of the pages' tokens once, q, out and lse
        lens = _sizes_of(c)
        rows = c["S"] * c["T"]
        keys = sum(lens)
        pages = sum(_pages(n, c["page"]) for n in lens)
        seen = sum(max(0, n - t) for n in lens for t in range(c["T"]))
        return {"bytes": 2 * keys * c["Hkv"] * c["d"] + pages * (4 + 2 * c["Hkv"]) + rows * c["Hq"] * (4 * c["d"] + 4),
                "flops": 4 * seen * c["Hq"] * c["d"]}
    prefix, tails = _sizes_of(c)
    rows = sum(sum(r) for r in tails)
    pairs = sum(sum(r) * p + sum(t * (t + 1) // 2 for t in r) for p, r in zip(prefix, tails))
    moved = 2 * sum(prefix) * c["Hkv"] * c["d"] + rows * (4 * c["Hq"] * c["d"] + 4 * c["Hkv"] * c["d"] + 4 * c["Hq"])
    return {"bytes": moved, "flops": 4 * pairs * c["Hq"] * c["d"]}


# ------------------------------------------------------------------------------------------ 64 bits
def _turned64(x, pos, rot, interleaved, freq, amplitude):
    """The rotation as a product of complex numbers."""
    turn = torch.polar(torch.full((pos.numel(), 1, rot // 2), float(amplitude), dtype=torch.float64, device=DEV),
                       (pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device=DEV)).unsqueeze(1))
    y = x.double().clone()
    i = torch.arange(rot // 2, device=DEV)
    at, to = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = torch.complex(y[..., at], y[..., to]) * turn
    y[..., at], y[..., to] = z.real, z.imag
    return y


def _e4m3(y):
    """The nearest value of four significant bits, exponent -6 and up, at most 448; ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_append(c, st):
    import numpy as np
    cache, page, Hkv = st["cache"], c["page"], c["Hkv"]
    new, start = _sizes_of(c)
    table = st["table"].cpu().numpy()
    freq, amplitude = _frequencies(c["rot"], "none")
    pos = torch.tensor(np.concatenate([np.arange(a, a + b) for a, b in zip(start, new)]), device=DEV)
    out = {}
    for name in ("k", "v"):
        x = st[name].double()
        if name == "k":
            x = _turned64(x, pos, c["rot"], c["interleaved"], freq, amplitude)
        codes = cache[name].double()
        scale = torch.exp2(cache[name + "_scale"].view(torch.uint8).double() - 127)
        row = 0
        for s in range(c["S"]):
            at, end = start[s], start[s] + new[s]
            while at < end:
                p = int(table[s, at // page])
                o, m = at % page, min(page - at % page, end - at)
                rows = x[row:row + m].transpose(0, 1)  # [Hkv, m, d]
                most = rows.abs().amax(dim=(1, 2))
                e = torch.ceil(torch.log2(most / 448)).clamp(E_MIN, E_MAX)
                sc = torch.exp2(torch.where(most <= 448 * torch.exp2(e - 1), e - 1, e).clamp(E_MIN, E_MAX))
                if o:
                    sc = torch.maximum(sc, scale[p])
                    codes[p, :, :o] = _e4m3(codes[p, :, :o] * (scale[p] / sc)[:, None, None])
                codes[p, :, o:o + m] = _e4m3(rows / sc[:, None, None])
                scale[p] = sc
                row, at = row + m, at + m
        out[name], out[name + "_scale"] = codes, scale
    return out


def _exact_token(c, st):
    S, T, Hq, Hkv, d, page = c["S"], c["T"], c["Hq"], c["Hkv"], c["d"], c["page"]
    lens = _sizes_of(c)
    out = torch.empty(S, T, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(Hq, S * T, dtype=torch.float64, device=DEV)
    for s in range(S):
        at = st["table"][s, :_pages(lens[s], page)].long()
        kv = []
        for name in ("k", "v"):
            x = st["cache"][name].view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
            x = x * torch.exp2(st["cache"][name + "_scale"].view(torch.uint8)[at].double() - 127)[..., None, None]
            kv.append(x.permute(1, 0, 2, 3).reshape(Hkv, -1, d).repeat_interleave(Hq // Hkv, dim=0))
        for t in range(T):
            n = lens[s] - (T - 1 - t)
            z = torch.einsum("hd,hnd->hn", st["q"][s, t].double(), kv[0][:, :n]) / math.sqrt(d)
            lse[:, s * T + t] = torch.logsumexp(z, dim=1)
            out[s, t] = torch.einsum("hn,hnd->hd", torch.softmax(z, dim=1), kv[1][:, :n])
    return {"out": out, "lse": lse}


def _exact_tail(c, st):
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    prefix, tails = _sizes_of(c)
    rows = st["q"].shape[0]
    out = torch.empty(rows, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(Hq, rows, dtype=torch.float64, device=DEV)
    row = 0
    for r, P in enumerate(prefix):
        at = st["table"][r, :_pages(P, page)].long()
        pre = []
        for name in ("k", "v"):
            x = st["cache"][name].view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
            x = x * torch.exp2(st["cache"][name + "_scale"].view(torch.uint8)[at].double() - 127)[..., None, None]
            pre.append(x.permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :P])
        for t in tails[r]:
            own_row = slice(row, row + t)
            later = torch.ones(t, t, dtype=torch.bool, device=DEV).triu(1)
            for h in range(Hkv):
                grp = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                k = torch.cat([pre[0][h], st["k"][own_row, h].double()])
                v = torch.cat([pre[1][h], st["v"][own_row, h].double()])
                z = torch.einsum("tgd,nd->gtn", st["q"][own_row, grp].double(), k) / math.sqrt(d)
                z[:, :, P:].masked_fill_(later, -math.inf)
                total = torch.logsumexp(z, dim=-1)
                lse[grp, own_row] = total
                out[own_row, grp] = torch.einsum("gtn,nd->tgd", torch.exp(z - total.unsqueeze(-1)), v)
            row += t
    return {"out": out, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        freq, amplitude = _frequencies(case["rot"], case["scaling"])
        return {x: _turned64(st[x], st["pos"], case["rot"], case["interleaved"], freq, amplitude) for x in ("q", "k")}
    return {"append": _exact_append, "token": _exact_token, "tail": _exact_tail}[case["op"]](case, st)
