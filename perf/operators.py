"""Measured calls of the cache-eviction and whole-vocabulary readout operators.

Three operators: the attention weight every cached prefix key received (``weights``), the eviction
of the lightest keys from a KV arena region (``evict``), and the log probabilities of given tokens
with entropy and top alternatives over the whole vocabulary (``logprobs``).  ``run`` computes them
with elementary torch operations in 32 bits, or, where ``own`` is true, through the library.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------ cases
def _weights(name, rows, P, Hq, Hkv, d, decay):
    return {"name": name, "op": "weights", "rows": rows, "P": P, "Hq": Hq, "Hkv": Hkv, "d": d, "decay": decay}


def _evict(name, P, keep, Hkv, d, sink, recent, seen):
    return {"name": name, "op": "evict", "P": P, "keep": keep, "Hkv": Hkv, "d": d, "sink": sink, "recent": recent,
            "seen": seen}


def _logprobs(name, n, H, V, T, top, gather):
    return {"name": name, "op": "logprobs", "n": n, "H": H, "V": V, "T": T, "top": top, "gather": gather}


def listed():
    return [
        # four short questions against a 64-token prompt: launch latency
        _weights("weights_tiny", 60, 64, 4, 2, 64, 0.0),
        # one token of one question against a long document, added to what the cache gathered before
        _weights("weights_one_token", 1, 18432, 32, 8, 128, 1.0),
        # sixteen questions against a 2k prompt
        _weights("weights_2k", 1275, 2048, 32, 8, 128, 0.0),
        # every question of the long-document workload, earlier weights fading
        _weights("weights_18k", 10240, 18432, 32, 8, 128, 0.5),
        # a short prompt cut to half
        _evict("evict_tiny", 64, 32, 2, 64, 4, 8, 64),
        # the long document cut to half
        _evict("evict_18k", 18432, 9216, 8, 128, 4, 256, 18432),
        # the longest prefix, already evicted once, cut to a quarter
        _evict("evict_max", 131072, 32768, 8, 128, 16, 1024, 200000),
        # a small model: launch latency
        _logprobs("logprobs_tiny", 4, 256, 1024, 1.0, 5, True),
        # the next token of one sequence, with the usual twenty alternatives
        _logprobs("logprobs_one_token", 1, 2560, 151936, 1.0, 20, False),
        # the answer position of every question of the long-document workload
        _logprobs("logprobs_18k", 64, 2560, 151936, 0.7, 8, True),
        # the answer positions of the largest request, wide model
        _logprobs("logprobs_max", 512, 5120, 151936, 1.0, 20, True),
        # a prompt scored token by token
        _logprobs("logprobs_prompt", 4096, 2560, 151936, 1.0, 5, False),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["weights", "evict", "logprobs"])
    if op == "weights":
        Hq, Hkv, d = rng.choice([(4, 2, 64), (32, 8, 128), (40, 8, 128), (8, 8, 64), (16, 2, 128), (5, 1, 64), (28, 4, 128)])
        P = _log_uniform(rng, 64, 131072)
        rows = _log_uniform(rng, 1, max(1, min(10240, 10240 * 18432 * 32 // (P * Hq))))
        c = _weights("", rows, P, Hq, Hkv, d, rng.choice([0.0, 0.5, 1.0]))
    elif op == "evict":
        P = _log_uniform(rng, 64, 131072)
        Hkv, d = rng.choice([(2, 64), (8, 128), (1, 64), (4, 128), (5, 64)])
        recent = rng.randint(0, P // 16)
        c = _evict("", P, max(1, int(P * rng.uniform(0.05, 0.5))), Hkv, d, rng.randint(0, 16), recent,
                   P + rng.choice([0, rng.randint(1, P)]))
    else:
        H = 8 * _log_uniform(rng, 32, 640)
        V = _log_uniform(rng, 1000, 151936)
        n = _log_uniform(rng, 1, max(1, min(4096, 4096 * 151936 * 2560 // (H * V))))
        c = _logprobs("", n, H, V, round(rng.uniform(0.5, 1.5), 3), rng.randint(0, 20), rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _prepare_weights(c, seed):
    g = _gen(seed)
    rows, P, Hq, Hkv, d = c["rows"], c["P"], c["Hq"], c["Hkv"], c["d"]
    q = torch.randn(rows, Hq, d, device=DEV, generator=g).to(torch.bfloat16)
    k = torch.randn(P, Hkv, d, device=DEV, generator=g).to(torch.bfloat16)
    # keys differ in how much attention they draw: a few stand out for every query
    k = (k.float() * (0.6 + 0.8 * torch.rand(P, Hkv, 1, device=DEV, generator=g))).to(torch.bfloat16)
    # the attention's log-sum-exp over the prefix; a question's own tail adds a little to it
    lse = torch.empty(Hq, rows, device=DEV)
    grp = Hq // Hkv
    for h in range(Hkv):
        step = max(1, (1 << 29) // P // grp)
        for a in range(0, rows, step):
            s = torch.einsum("tgd,pd->gtp", q[a:a + step, h * grp:(h + 1) * grp], k[:, h]).float() / math.sqrt(d)
            lse[h * grp:(h + 1) * grp, a:a + step] = torch.logsumexp(s, dim=-1)
    lse += 0.1 * torch.rand(Hq, rows, device=DEV, generator=g)
    prev = torch.rand(Hkv, P, device=DEV, generator=g) * (2.0 * rows * grp / P) if c["decay"] else None
    st = {"q": q, "k": k, "lse": lse, "prev": prev}
    if own:
        from shared_prefix_question_gb300 import blink
        st["ws"] = blink.new_workspace(blink.key_weights_workspace_bytes(rows, P, Hq, Hkv, d), DEV)
    return st


def _prepare_evict(c, seed):
    g = _gen(seed)
    P, Hkv, d, keep = c["P"], c["Hkv"], c["d"], c["keep"]
    # accumulated attention is heavy-tailed, and keys that nothing attends to have underflowed to zero
    w = torch.exp(2.0 * torch.randn(Hkv, P, device=DEV, generator=g))
    w = torch.where(torch.rand(Hkv, P, device=DEV, generator=g) < 0.03, torch.zeros_like(w), w)
    k = torch.randn(P, Hkv, d, device=DEV, generator=g).to(torch.bfloat16)
    v = torch.randn(P, Hkv, d, device=DEV, generator=g).to(torch.bfloat16)
    if c["seen"] > P:  # evicted before: each head holds P of the positions seen, in any order
        pos = torch.stack([torch.randperm(c["seen"], device=DEV, generator=g)[:P] for _ in range(Hkv)]).to(torch.int32)
    else:
        pos = torch.arange(P, device=DEV, dtype=torch.int32).repeat(Hkv, 1)
    st = {"w": w, "k": k, "v": v, "pos": pos, "k_dst": torch.zeros(keep, Hkv, d, dtype=torch.bfloat16, device=DEV),
          "v_dst": torch.zeros(keep, Hkv, d, dtype=torch.bfloat16, device=DEV)}
    if own:
        from shared_prefix_question_gb300 import blink
        st["ws"] = blink.new_workspace(blink.kv_evict_workspace_bytes(P, keep, Hkv), DEV)
    return st


def _prepare_logprobs(c, seed):
    g = _gen(seed)
    n, H, V = c["n"], c["H"], c["V"]
    W = torch.empty(V, H, dtype=torch.bfloat16, device=DEV)
    for a in range(0, V, 1 << 14):
        b = min(V, a + (1 << 14))
        W[a:b] = (0.02 * math.sqrt(2560 / H) * torch.randn(b - a, H, device=DEV, generator=g)).to(torch.bfloat16)
    # a trained model's distribution is peaked: a few dozen tokens stand out, each a step below the
    # one before, over a floor of noise.  The hidden state is the noise plus the combination of
    # those tokens' rows that gives them these logits.
    m = 24
    hid = torch.randn(n, H, device=DEV, generator=g)
    ids = torch.randint(0, V - V % m, (n, m), device=DEV, generator=g) // m * m + torch.arange(m, device=DEV)
    ids = torch.gather(ids, 1, torch.rand(n, m, device=DEV, generator=g).argsort(1))
    first = 9.0 + 7.0 * torch.rand(n, 1, device=DEV, generator=g)
    want = first - 0.15 * torch.arange(m, device=DEV) - 0.05 * torch.rand(n, m, device=DEV, generator=g)
    for a in range(0, n, 512):
        rowsW = W[ids[a:a + 512]].float()
        lack = want[a:a + 512] - torch.einsum("nmh,nh->nm", rowsW, hid[a:a + 512])
        coef = torch.linalg.solve(torch.einsum("nmh,nkh->nmk", rowsW, rowsW), lack)
        hid[a:a + 512] += torch.einsum("nm,nmh->nh", coef, rowsW)
    # the given token: usually one of the likely ones, sometimes any
    t = torch.gather(ids, 1, torch.randint(0, m, (n, 1), device=DEV, generator=g)).squeeze(1)
    t = torch.where(torch.rand(n, device=DEV, generator=g) < 0.25,
                    torch.randint(0, V, (n,), device=DEV, generator=g), t).to(torch.int32)
    hid = hid.to(torch.bfloat16)
    if c["gather"]:  # answer positions scattered over the tail rows
        rows = 3 * n + 5
        idx = torch.randperm(rows, device=DEV, generator=g)[:n]
        full = torch.randn(rows, H, device=DEV, generator=g).to(torch.bfloat16)
        full[idx] = hid
        hid, idx = full, idx.to(torch.int32)
    else:
        idx = None
    st = {"hidden": hid, "idx": idx, "W": W, "targets": t, "T": c["T"], "top": c["top"]}
    if own:
        from shared_prefix_question_gb300 import blink
        st["ws"] = blink.new_workspace(blink.token_logprobs_workspace_bytes(n, H, V, c["top"]), DEV)
    return st


def prepare(case, seed):
    st = {"weights": _prepare_weights, "evict": _prepare_evict, "logprobs": _prepare_logprobs}[case["op"]](case, seed)
    st["case"] = case
    return st


# ------------------------------------------------------------------------------------------ passes
def _run_weights(st):
    c = st["case"]
    if own:
        from shared_prefix_question_gb300 import blink
        w, _ = blink.blink_prefix_key_weights(st["q"], st["k"], st["lse"], prev=st["prev"], decay=c["decay"], ws=st["ws"])
        return {"weights": w}
    rows, P, Hq, Hkv, d = c["rows"], c["P"], c["Hq"], c["Hkv"], c["d"]
    qt = st["q"].float().view(rows, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
    s = torch.bmm(qt, st["k"].float().permute(1, 2, 0))  # [Hkv, g * rows, P]
    s.mul_(1.0 / math.sqrt(d)).sub_(st["lse"].view(Hkv, -1, 1)).exp_()
    w = s.sum(dim=1)
    if c["decay"]:
        w = w + c["decay"] * st["prev"]
    return {"weights": w}


def _run_evict(st):
    c = st["case"]
    P, keep, seen = c["P"], c["keep"], c["seen"]
    if own:
        from shared_prefix_question_gb300 import blink
        r = blink.blink_kv_evict(st["w"], st["k"], st["v"], keep, pos=st["pos"], sink=c["sink"],
                                 recent_from=seen - c["recent"], k_dst=st["k_dst"], v_dst=st["v_dst"], ws=st["ws"])
        return {"slots": r["slots"], "k": st["k_dst"], "v": st["v_dst"], "weights": r["weights"], "pos": r["pos"]}
    w, pos = st["w"], st["pos"]
    slot = torch.arange(P, device=w.device)
    safe = (pos < c["sink"]) | (pos >= seen - c["recent"])
    by_weight = torch.sort(w, dim=1, descending=True, stable=True).indices
    by_class = torch.sort(torch.gather(safe.to(torch.int32), 1, by_weight), dim=1, descending=True, stable=True).indices
    kept = torch.zeros_like(safe).scatter_(1, torch.gather(by_weight, 1, by_class)[:, :keep], True)
    # kept slots below `keep` stay; the others below it take the kept slots from `keep` on, in order
    low, high = kept[:, :keep], kept[:, keep:]
    n_in = high.sum(dim=1, keepdim=True)
    order = torch.sort((~high).to(torch.int32), dim=1, stable=True).indices + keep  # kept ones first, ascending
    rank = (torch.cumsum((~low).to(torch.int64), dim=1) - 1).clamp(min=0)
    rank = torch.minimum(rank, (n_in - 1).clamp(min=0))
    slots = torch.where(low, slot[:keep].expand_as(low), torch.gather(order, 1, rank))
    row = slots.t().unsqueeze(-1).expand(-1, -1, c["d"])
    st["k_dst"].copy_(torch.gather(st["k"], 0, row))
    st["v_dst"].copy_(torch.gather(st["v"], 0, row))
    return {"slots": slots.to(torch.int32), "k": st["k_dst"], "v": st["v_dst"], "weights": torch.gather(w, 1, slots),
            "pos": torch.gather(pos, 1, slots)}


def _run_logprobs(st):
    if own:
        from shared_prefix_question_gb300 import blink
        r = blink.blink_token_logprobs(st["hidden"], st["W"], targets=st["targets"], row_idx=st["idx"],
                                       temperature=st["T"], top=st["top"], ws=st["ws"])
        return {k: r[k] for k in ("logprob", "entropy", "lse", "top_ids", "top_logprobs") if r[k] is not None}
    h = st["hidden"] if st["idx"] is None else st["hidden"][st["idx"].long()]
    z = torch.mm(h.float(), st["W"].float().t())
    z.mul_(1.0 / st["T"])
    best = z.max(dim=1, keepdim=True).values
    lse = best + (z - best).exp_().sum(dim=1, keepdim=True).log()
    out = {"logprob": (torch.gather(z, 1, st["targets"].long().unsqueeze(1)) - lse).squeeze(1), "lse": lse.squeeze(1)}
    if st["top"]:
        top = torch.topk(z, st["top"], dim=1)
        out["top_ids"] = top.indices.to(torch.int32)
        out["top_logprobs"] = top.values - lse
    lp = z.sub_(lse)
    out["entropy"] = -(lp.exp() * lp).sum(dim=1)
    return out


def run(state):
    return {"weights": _run_weights, "evict": _run_evict, "logprobs": _run_logprobs}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "weights":
        moved = 2 * c["rows"] * c["Hq"] * c["d"] + 2 * c["P"] * c["Hkv"] * c["d"] + 4 * c["rows"] * c["Hq"]
        moved += 4 * c["Hkv"] * c["P"] * (2 if c["decay"] else 1)
        return {"bytes": moved, "flops": 2 * c["rows"] * c["Hq"] * c["P"] * c["d"]}
    if c["op"] == "evict":
        row = 2 * 2 * c["d"] + 4 + 4  # K and V, the weight, the position
        return {"bytes": c["Hkv"] * (8 * c["P"] + c["keep"] * (4 * c["d"] + row + 4)), "flops": 0}
    moved = 2 * c["V"] * c["H"] + 2 * c["n"] * c["H"] + c["n"] * (4 + 4 * 3 + 8 * c["top"])
    return {"bytes": moved, "flops": 2 * c["n"] * c["V"] * c["H"]}


# ------------------------------------------------------------------------------------------ 64 bits
def _exact_weights(c, st):
    rows, P, Hq, Hkv, d = c["rows"], c["P"], c["Hq"], c["Hkv"], c["d"]
    w = torch.zeros(Hkv, P, dtype=torch.float64, device=DEV)
    step = max(1, (1 << 28) // P)
    for hq in range(Hq):
        kt = st["k"][:, hq // (Hq // Hkv)].double().t().contiguous()
        for a in range(0, rows, step):
            s = st["q"][a:a + step, hq].double() @ kt
            w[hq // (Hq // Hkv)] += torch.exp(s / math.sqrt(d) - st["lse"][hq, a:a + step, None].double()).sum(0)
    if c["decay"]:
        w += c["decay"] * st["prev"].double()
    return {"weights": w}


def _exact_evict(c, st):
    import numpy as np
    P, keep, Hkv = c["P"], c["keep"], c["Hkv"]
    w, pos = st["w"].double().cpu().numpy(), st["pos"].cpu().numpy()
    slots = np.empty((Hkv, keep), np.int32)
    for h in range(Hkv):
        guarded = (pos[h] < c["sink"]) | (pos[h] >= c["seen"] - c["recent"])
        kept = np.sort(np.lexsort((np.arange(P), -w[h], ~guarded))[:keep])
        slots[h] = np.arange(keep)
        holes = np.setdiff1d(np.arange(keep), kept[kept < keep])
        slots[h, holes] = kept[kept >= keep]
    s = torch.from_numpy(slots).to(DEV).long()
    head = torch.arange(Hkv, device=DEV)
    return {"slots": s.to(torch.int32), "k": st["k"][s.t(), head].double(), "v": st["v"][s.t(), head].double(),
            "weights": st["w"].double()[head[:, None], s], "pos": st["pos"][head[:, None], s]}


def _exact_logprobs(c, st):
    parts = {k: [] for k in ("logprob", "entropy", "lse", "top_ids", "top_logprobs")}
    Wt = st["W"].double().t()
    for a in range(0, c["n"], 256):
        idx = torch.arange(a, min(c["n"], a + 256), device=DEV)
        z = st["hidden"][idx if st["idx"] is None else st["idx"].long()[idx]].double() @ Wt / c["T"]
        lse = torch.logsumexp(z, dim=1)
        p = torch.exp(z - lse[:, None])
        parts["logprob"].append(z[torch.arange(len(idx), device=DEV), st["targets"].long()[idx]] - lse)
        parts["entropy"].append((p * (lse[:, None] - z)).sum(1))
        parts["lse"].append(lse)
        val, at = torch.sort(z, dim=1, descending=True, stable=True)
        parts["top_ids"].append(at[:, :c["top"]].to(torch.int32))
        parts["top_logprobs"].append(val[:, :c["top"]] - lse[:, None])
    return {k: torch.cat(v) for k, v in parts.items() if c["top"] or not k.startswith("top")}


def exact(case, seed):
    st = prepare(case, seed)
    return {"weights": _exact_weights, "evict": _exact_evict, "logprobs": _exact_logprobs}[case["op"]](case, st)
