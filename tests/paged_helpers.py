"""Plain 64-bit forms of the rotary, append and paged-attention calls, and caches to call them on."""
from __future__ import annotations

import math

import torch

DEV = "cuda"
BF16, F16, F32, E4M3 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24, 2.0 ** -4  # half a step, relative to the value


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def frequencies(rot, base, scaling=None, factor=1.0, original=0, low=0.0, high=0.0):
    """theta_i and the amplitude, from the formulas."""
    n = rot // 2
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    theta = [base ** (-2 * i / rot) for i in range(n)]
    if scaling == "linear":
        theta = [t / factor for t in theta]
    if scaling == "by_dim":
        at = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(high))), min(rot - 1, math.ceil(at(low)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(n)]
        return [t * (1 - r) + t / factor * r for t, r in zip(theta, ramp)], 0.1 * math.log(factor) + 1
    if scaling == "by_turns":
        for i, t in enumerate(theta):
            keep = min(1.0, max(0.0, (original * t / (2 * math.pi) - low) / (high - low)))
            theta[i] = keep * t + (1 - keep) * t / factor
    return theta, 1.0


def rotate(x, pos, theta, amplitude, interleaved):
    """x [n, H, d] in 64 bits; also the size that 32-bit roundings are relative to (|x0| + |x1| of a pair)."""
    rot = 2 * len(theta)
    y = x.double().clone()
    size = y.abs()
    angle = pos.double()[:, None, None] * torch.tensor(theta, dtype=torch.float64, device=x.device)
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    x0, x1 = y[..., a], y[..., b]
    y[..., a], y[..., b] = (amplitude * (x0 * angle.cos() - x1 * angle.sin()), amplitude * (x0 * angle.sin() + x1 * angle.cos()))
    size[..., a] = size[..., b] = amplitude * (x0.abs() + x1.abs())
    return y, size


def e4m3(y):
    """Nearest e4m3 value, ties to even, at most 448; NaN stays."""
    y = y.clamp(-512, 512)  # infinities too
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    r = torch.round(y / step) * step
    return torch.where(y.isnan(), y, r.clamp(-448, 448))


def scale_exponent(m):
    """The smallest e in -48..32 with m <= 448 * 2^e."""
    e = -48
    while e < 32 and m > 448.0 * 2.0 ** e:
        e += 1
    return e


def new_cache(g, n_pages, Hkv, page, d, fused=False, spread=0, filler=0x7F):
    """A cache whose every slot holds `filler` (0x7F: NaN) and whose scales are arbitrary; `fused`: K and V are halves of one tensor."""
    if fused:
        both = torch.full((n_pages, 2, Hkv, page, d), filler, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        k, v = both[:, 0], both[:, 1]
        s = torch.full((n_pages, 2, Hkv + 3), 120, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
        ks, vs = s[:, 0, :Hkv], s[:, 1, :Hkv]
    else:
        k, v = (torch.full((n_pages, Hkv, page, d), filler, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.full((n_pages, Hkv), 120, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu) for _ in range(2))
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}


def table_for(g, lens, page, extra=2, width=None):
    """Pages for sequences of `lens` tokens, in any order; -1 behind them.  (table, number of pages)."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + extra
    perm = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    table = torch.full((len(lens), width or max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    return table, total


def fill(g, cache, table, lens, k_exp=(-8, -5), v_exp=(-8, -5)):
    """Random codes and scales in the slots that the sequences hold, others left as they are."""
    Hkv, page, d = cache["k"].shape[1:]
    for s, n in enumerate(lens):
        for i in range(-(-n // page)):
            p, m = int(table[s, i]), min(page, n - i * page)
            for name, (lo, hi) in (("k", k_exp), ("v", v_exp)):
                x = (110 * randn(g, Hkv, m, d)).clamp(-448, 448).to(torch.float8_e4m3fn)
                cache[name].view(torch.uint8)[p, :, :m] = x.view(torch.uint8)
                cache[name + "_scale"].view(torch.uint8)[p] = (127 + torch.randint(lo, hi + 1, (Hkv,), device=DEV, generator=g)).to(torch.uint8)


def values(cache, name, table_row, n):
    """[Hkv, n, d] in 64 bits: the first n tokens of a sequence."""
    page = cache[name].shape[2]
    at = table_row[:-(-n // page)].long()
    x = cache[name].view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
    x = x * torch.exp2(cache[name + "_scale"].view(torch.uint8)[at].double() - 127)[..., None, None]
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def attend(q, k, v, scale):
    """One row: q [Hq, d] over k, v [Hkv, n, d]: (out, lse, what roundings of its weights can change, largest sum of
    |q k|), 64 bits.  A weight is rounded to fp16: half a step of itself, or 2^-25 of the largest weight."""
    Hq, d = q.shape
    Hkv, n = k.shape[:2]
    if n == 0:
        z = torch.zeros(Hq, d, dtype=torch.float64, device=q.device)
        return z, torch.full((Hq,), -math.inf, dtype=torch.float64, device=q.device), torch.stack([z, z]), torch.zeros(Hq, dtype=torch.float64, device=q.device)
    k, v = (x.repeat_interleave(Hq // Hkv, dim=0) for x in (k, v))
    z = torch.einsum("hd,hnd->hn", q.double(), k) * scale
    lse = torch.logsumexp(z, dim=1)
    w = torch.exp(z - lse[:, None])
    size = torch.einsum("hd,hnd->hn", q.double().abs(), k.abs()).amax(dim=1) * scale
    return torch.einsum("hn,hnd->hd", w, v), lse, torch.stack([torch.einsum("hn,hnd->hd", w, v.abs()), v.abs().sum(dim=1)]), size


def token_reference(q, cache, table, lens, scale=0.0):
    S, T, Hq, d = q.shape
    scale = scale or 1 / math.sqrt(d)
    out = torch.empty(S, T, Hq, d, dtype=torch.float64, device=DEV)
    mag = torch.empty(2, S, T, Hq, d, dtype=torch.float64, device=DEV)
    lse, size = (torch.empty(Hq, S, T, dtype=torch.float64, device=DEV) for _ in range(2))
    for s, n in enumerate(lens):
        k, v = values(cache, "k", table[s], n), values(cache, "v", table[s], n)
        for t in range(T):
            m = max(0, n - (T - 1 - t))
            out[s, t], lse[:, s, t], mag[:, s, t], size[:, s, t] = attend(q[s, t], k[:, :m], v[:, :m], scale)
    return out, lse.reshape(Hq, S * T), mag, size.reshape(Hq, S * T)


def check_attention(out, lse, ref):
    """Against the plain form.  A score is a sum of exact products, its roundings (the tensor core's sums, the scale, the
    reduction) at most 64 half steps of 32 bits of the largest sum of |q k|; the exponential and the sums add some
    2^-22 each.  The second product adds up to 64 partial sums, each cut off at 2^-23.  The output is rounded to bf16."""
    want, want_lse, mag, size = ref
    none = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, none)
    x = (64 * F32 * size + 2.0 ** -20)  # relative error of a weight, absolute of lse
    live = ~none
    assert bool(((lse.double() - want_lse).abs()[live] <= (x + 4 * F32 * want_lse.abs())[live]).all())
    S, T, Hq, d = want.shape
    xr = x.reshape(Hq, S, T).permute(1, 2, 0)[..., None]
    bound = BF16 * want.abs() + (F16 + 2 * xr + 2.0 ** -17) * mag[0] + 2.0 ** -25 * mag[1] + 2.0 ** -126
    err = (out.double() - want).abs()
    assert bool(out.isfinite().all())
    assert bool((err <= bound).all()), f"largest excess {(err - bound).max():.3e}, error {err.max():.3e}"
