"""Plain float64 forms (torch on the CPU) of the losses over the vocabulary and
of AdamW, with the errors that fp32 arithmetic may make, for the tests."""

from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32, relative


def half_step(ref: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """Rounding of values to `dtype` once (and the smallest step's half)."""
    return ref.abs() * (torch.finfo(dtype).eps / 2) + {torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}.get(dtype, 0.0)


# ------------------------------------------------------------------ losses --

def logprob(logits, targets, vocab, tau):
    """(logp, lse, their bound): float64; rows without a token are zeros.

    Bound: a term's exponent is off by three roundings (the difference, the
    factor, the product), its exponential by 2^-22; a term with exponent -d has
    weight e^-d, and d e^-d summed over the weights is at most ln V + 1.  The
    sum of V positive terms, at most V / 256 + 64 of them in a row (at least 32
    threads, eight a granule, four granules at a time), each rescaled at most
    once a granule and once a joining: 2^-22 each.  The logarithm and the last
    differences: four roundings of their magnitudes."""
    x = logits.cpu().double().reshape(-1, logits.shape[-1])[:, :vocab] / tau
    t = targets.cpu().reshape(-1)
    has = t >= 0
    m = x.max(1).values
    lse = m + torch.log(torch.exp(x - m[:, None]).sum(1))
    xa = x.gather(1, t.clamp(min=0, max=vocab - 1)[:, None])[:, 0]
    logp = xa - lse
    rel = (vocab / 256 + 64) * 2.0 ** -22 + 3 * U * (math.log(vocab) + 1)
    tol = rel + 4 * U * ((xa - m).abs() + math.log(vocab) + 1)
    zero = torch.zeros_like(logp)
    return torch.where(has, logp, zero), torch.where(has, lse, zero), tol, tol + 4 * U * m.abs()


def softmax_grad(logits, targets, coef, tol_coef, vocab, tau, lse, tol_lse):
    """(dlogits, bound) in float64 from the gradient `coef` at logp, itself
    off by tol_coef; p's exponent is off by tol_lse and three roundings, and an
    exponential below 2^-126 may be taken as 0."""
    n = logits.shape[-1]
    x = logits.cpu().double().reshape(-1, n)
    t = targets.cpu().reshape(-1)
    p = torch.zeros_like(x)
    d = x[:, :vocab] / tau - lse[:, None]
    p[:, :vocab] = torch.exp(d)
    hot = torch.zeros_like(x)
    hot.scatter_(1, t.clamp(min=0)[:, None], 1.0)
    on = ((t >= 0) & (coef != 0))[:, None]
    c = (coef / tau)[:, None]
    ref = torch.where(on, c * (hot - p), torch.zeros_like(x))
    rel = torch.zeros_like(x)
    rel[:, :vocab] = tol_lse[:, None] + 4 * U * d.abs() + 2.0 ** -21
    tol = c.abs() * (p * rel + 2 * U * hot + 2.0 ** -126) + (tol_coef / tau)[:, None] * (hot + p)
    return ref, torch.where(on, tol, torch.zeros_like(tol)) + half_step(ref, logits.dtype)


def policy(logits, targets, old, adv, weights, ref, lo, hi, kl, vocab, tau, scale=1.0):
    """float64 forms and bounds: dict of (value, bound)."""
    logp, lse, tol, tol_lse = logprob(logits, targets, vocab, tau)
    w, a, o = (z.cpu().double().reshape(-1) for z in (weights, adv, old))
    on = (w != 0) & (targets.cpu().reshape(-1) >= 0)
    zero = torch.zeros_like(logp)
    r = torch.exp(logp - o)
    free, held = r * a, r.clamp(1 - lo, 1 + hi) * a
    tol_r = r * (tol + 4 * U * (logp - o).abs() + 2.0 ** -21)
    loss, slope = -torch.minimum(free, held), torch.where(free <= held, -free, zero)
    tol_loss, tol_slope = tol_r * a.abs() + 4 * U * free.abs(), tol_r * a.abs() + 4 * U * free.abs()
    if kl:
        d = ref.cpu().double().reshape(-1) - logp
        e = torch.exp(d)
        off = (e + 1) * (tol + 2 * U * d.abs()) + 2.0 ** -21 * ((e - 1).abs() + d.abs())
        loss, slope = loss + kl * (e - 1 - d), slope - kl * (e - 1)
        tol_loss, tol_slope = tol_loss + kl * off, tol_slope + kl * off
    loss, slope = torch.where(on, w * loss, zero), torch.where(on, w * slope, zero)
    tol_loss = torch.where(on, w.abs() * tol_loss, zero) + 2 * U * loss.abs()
    tol_slope = torch.where(on, w.abs() * tol_slope, zero) + 4 * U * slope.abs()
    d, tol_d = softmax_grad(logits, targets, slope * scale, tol_slope * abs(scale), vocab, tau, lse, tol_lse)
    return {"token_loss": (loss, tol_loss), "logp": (torch.where(on, logp, zero), tol),
            "loss": (loss.sum(), tol_loss.sum() + 2 * U * loss.sum().abs()), "dlogits": (d, tol_d)}


def preference(logits, targets, offsets, ref, beta, ls, mean, vocab, tau, scale=1.0):
    logp, lse, tol, tol_lse = logprob(logits, targets, vocab, tau)
    t = targets.cpu().reshape(-1)
    T = len(t)
    at = offsets.cpu().clamp(0, T).tolist()
    inside = torch.zeros(T, dtype=torch.bool)
    inside[at[0]:at[-1]] = True
    on = (t >= 0) & inside
    zero = torch.zeros_like(logp)
    gap = torch.where(on, logp - (0 if ref is None else ref.cpu().double().reshape(-1)), zero)
    off = torch.where(on, tol, zero)
    s, ds, count = [], [], []
    for a, b in zip(at, at[1:]):
        n = max(1, int(on[a:b].sum())) if mean else 1
        count.append(n)
        s.append(gap[a:b].sum() / n)
        ds.append(off[a:b].sum() / n)
    s, ds = torch.stack(s), torch.stack(ds)
    z = beta * (s[0::2] - s[1::2])
    dz = abs(beta) * (ds[0::2] + ds[1::2]) + 4 * U * z.abs()
    sp = torch.nn.functional.softplus
    per = (1 - ls) * sp(-z) + ls * sp(z)
    loss, dloss = per.mean(), (dz + 8 * U * per).mean()
    slope = (ls * torch.sigmoid(z) - (1 - ls) * torch.sigmoid(-z)) * beta / len(z)
    dslope = abs(beta) / len(z) * (dz / 4 + 2.0 ** -20)
    coef, dcoef = zero.clone(), zero.clone()
    for i, (a, b) in enumerate(zip(at, at[1:])):
        coef[a:b] = (slope[i // 2] if i % 2 == 0 else -slope[i // 2]) / count[i]
        dcoef[a:b] = dslope[i // 2] / count[i] if torch.is_tensor(dslope) and dslope.dim() else dslope
    coef, dcoef = torch.where(on, coef, zero), torch.where(on, dcoef, zero)
    d, tol_d = softmax_grad(logits, targets, coef * scale, dcoef * abs(scale), vocab, tau, lse, tol_lse)
    return {"loss": (loss, dloss), "margin": (z, dz), "logratio": (s, ds + 2 * U * s.abs()),
            "logp": (torch.where(on, logp, zero), tol), "dlogits": (d, tol_d)}


# ------------------------------------------------------------------- AdamW --

def mix(x: np.ndarray) -> np.ndarray:
    m = np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x9E3779B1)) & m
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x85A308D3)) & m
    return x ^ (x >> np.uint64(16))


def bits_of(n: int, tensor: int, step: int, seed: int, first: int = 0) -> np.ndarray:
    """The hash of elements first .. first + n - 1 of a tensor in step + 1."""
    u = lambda v: np.array([v & 0xFFFFFFFF], dtype=np.uint64)
    k = mix(u(seed))
    for word in (seed >> 32, step, tensor):
        k = mix(k ^ u(word))
    e = np.arange(first, first + n, dtype=np.uint64)
    high = e >> np.uint64(32)
    key = np.where(high == 0, k, mix(k ^ high))
    return mix((((e & np.uint64(0xFFFFFFFF)) * np.uint64(0x13198A2F)) & np.uint64(0xFFFFFFFF)) ^ key)


def pad(x: torch.Tensor) -> torch.Tensor:
    n = x.numel()
    return torch.nn.functional.pad(x.reshape(-1), (0, -(-n // 128) * 128 - n)).view(-1, 128)


def e4m3_step(y: torch.Tensor) -> torch.Tensor:
    _, e = torch.frexp(y)
    return torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)


def code_range(x: torch.Tensor, tol: torch.Tensor, bits: np.ndarray, least: bool):
    """Smallest and largest value that |x|, off by at most tol (both
    float64 [n]), may be held as, with each block's multiplier and its bound.
    Two more roundings of the scaled value, and the one of its sum with 2^-6."""
    n = x.numel()
    top, off = pad(x.abs()).max(1, keepdim=True).values, pad(tol).max(1, keepdim=True).values
    scale = torch.where(top < 2.0 ** -100, torch.ones_like(top), top / 448)
    dscale = torch.where(top < 2.0 ** -100, torch.zeros_like(top), off / 448 + 2 * U * scale)
    y = pad(x.abs()) / scale
    dy = pad(tol) / scale + y * (dscale / scale + 4 * U) + 2.0 ** -29
    u = pad(torch.from_numpy(bits.astype(np.float64)))

    def held(v):
        v = v.clamp(min=0, max=448)
        step = e4m3_step(v)
        q = (torch.floor(v / step + (u + 0.5) / 65536) * step).clamp(max=448)
        if least:
            q = torch.where((v > 0) & (q == 0) & (top >= 2.0 ** -100), torch.full_like(q, 2.0 ** -9), q)
        return torch.where(top < 2.0 ** -100, torch.zeros_like(q), q)

    flat = lambda v: v.reshape(-1)[:n]
    return flat(held(y - dy)), flat(held(y + dy)), scale[:, 0], dscale[:, 0]


def adamw(p, g, m, v, t, lr, wd, b1, b2, eps, coef=1.0, tol_coef=0.0):
    """float64 [n] -> (p, m, v) and their bounds; t: the step being done.

    m and v: three roundings of each term; v's square doubles g's.  The update
    divides by sqrt(v): half of v's error, and ten roundings (the root, the bias
    corrections' expm1 and rsqrt, the quotient by reciprocal)."""
    g = g * coef
    dg = g.abs() * (tol_coef + 2 * U)
    mn, vn = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    dm = 3 * U * (b1 * m.abs() + (1 - b1) * g.abs()) + (1 - b1) * dg
    dv = 3 * U * (b2 * v + (1 - b2) * g * g) + 2 * (1 - b2) * g.abs() * dg + 2.0 ** -148
    root = vn.sqrt()
    den = root / math.sqrt(1 - b2 ** t) + eps
    upd = mn / (1 - b1 ** t) / den
    droot = torch.where(vn > 0, dv / root.clamp(min=1e-300), dv.sqrt())
    dupd = dm / (1 - b1 ** t) / den + upd.abs() * (droot / math.sqrt(1 - b2 ** t) / den + 24 * U)
    pn = p - lr * (wd * p + upd)
    dp = 2 * U * (p.abs() + pn.abs()) + lr * (dupd + 4 * U * (wd * p.abs() + upd.abs()))
    return (pn, dp), (mn, dm), (vn, dv), (root, droot + 2 * U * root)
