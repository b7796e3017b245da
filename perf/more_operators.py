"""Cases, plain forms and 64-bit values of the operators at the two ends of a
training step: the losses over the vocabulary with their gradients, and the
optimizer.

Operators (``case["op"]``), logits [T, n] of which the first v columns count:

* ``logprob``: log probability of each row's target, and the log of the sum.
* ``logprob_grad``: the gradient at the logits from the one at the log
  probabilities.
* ``policy``: clipped policy loss with a KL term, its gradient at the logits.
* ``preference``: loss of paired sequences' log ratios, its gradient likewise.
* ``adamw``: one AdamW step over many tensors, states in 32 or in 8 bits,
  gradients fp32, bf16 or FP8 (E4M3 codes and an fp32 multiplier per block of
  128), after clipping by the norm of all of them where ``clip``.

States in 8 bits are E4M3 codes of m and of r = sqrt(v) with a multiplier per
block of 128, rounded up with the probability of the rest: by 16 bits of a
hash of the element, its tensor, the step and a seed.
"""

import math
import random

import torch

own = False

TAU = 0.8                # the temperature of the losses' cases
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
LR, BETA1, BETA2, ADAM_EPS, MAX_NORM = 2e-5, 0.9, 0.95, 1e-8, 1.0
STEP0 = 1000             # steps that the optimizer has done


def listed():
    return [
        # one token scored, padded vocabulary: latency
        {"name": "logprob_1_50304", "op": "logprob", "t": 1, "v": 50257, "n": 50304, "dt": "bf16"},
        # a batch scored by the reference policy, rows that start anywhere
        {"name": "logprob_4096_50257", "op": "logprob", "t": 4096, "v": 50257, "n": 50257, "dt": "bf16"},
        # a few rows of a large vocabulary backward
        {"name": "logprob_grad_37_128001", "op": "logprob_grad", "t": 37, "v": 128001, "n": 128001, "dt": "bf16"},
        # a batch of fp32 logits backward
        {"name": "logprob_grad_2048_32000_f32", "op": "logprob_grad", "t": 2048, "v": 32000, "n": 32000, "dt": "f32"},
        # one sampled token
        {"name": "policy_1_50304", "op": "policy", "t": 1, "v": 50257, "n": 50304, "dt": "bf16", "kl": 0.05},
        # odd sizes in fp32
        {"name": "policy_1021_32003_f32", "op": "policy", "t": 1021, "v": 32003, "n": 32003, "dt": "f32", "kl": 0.05},
        # the tokens of a training step, the largest of the losses
        {"name": "policy_8192_50304", "op": "policy", "t": 8192, "v": 50257, "n": 50304, "dt": "bf16", "kl": 0.0},
        # one short pair
        {"name": "preference_1x24_32000", "op": "preference", "pairs": 1, "longest": 24, "tail": 3, "v": 32000,
         "n": 32000, "dt": "bf16", "ls": 0.0, "mean": False},
        # eight pairs of up to 500 tokens
        {"name": "preference_8x500_50304", "op": "preference", "pairs": 8, "longest": 500, "tail": 77, "v": 50257,
         "n": 50304, "dt": "bf16", "ls": 0.1, "mean": False},
        # the gains and a small projection: latency
        {"name": "adamw8_3_20000_f32", "op": "adamw", "count": 3, "total": 20000, "bits": 8, "grad": "f32",
         "clip": False},
        # many tensors of all sizes, states in 32 bits
        {"name": "adamw32_292_60M_bf16", "op": "adamw", "count": 292, "total": 60000000, "bits": 32, "grad": "bf16",
         "clip": True},
        # a GPT-6.7B layer's weights with their FP8 main gradients, the largest
        {"name": "adamw8_8_201M_fp8", "op": "adamw", "count": 8, "total": 201334784, "bits": 8, "grad": "fp8",
         "clip": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("logprob", "logprob_grad", "policy", "policy", "preference", "preference", "adamw", "adamw"))
    if op == "adamw":
        bits = rng.choice((8, 32))
        total = _log(rng, 1000, 180000000 if bits == 8 else 90000000)
        return {"op": op, "count": _log(rng, 1, min(500, total // 10)), "total": total, "bits": bits,
                "grad": rng.choice(("f32", "bf16", "fp8")), "clip": rng.random() < 0.6}
    v = _log(rng, 512, 131072)
    case = {"op": op, "v": v, "n": v if rng.random() < 0.5 else -(-v // 128) * 128,
            "dt": rng.choice(("bf16", "bf16", "f32"))}
    rows = min(8192, (400000000 if case["dt"] == "bf16" else 200000000) // case["n"])
    if op == "preference":
        case["pairs"] = _log(rng, 1, 32)
        case["longest"] = _log(rng, 1, min(2048, rows * 5 // 6 // (2 * case["pairs"])))
        return case | {"tail": rng.choice((0, 1, 50)), "ls": rng.choice((0.0, 0.1)), "mean": rng.random() < 0.3}
    case["t"] = _log(rng, 1, rows)
    if op == "policy":
        case["kl"] = rng.choice((0.0, 0.05))
    return case


# ------------------------------------------------------------------ inputs --

def _lengths(case):
    """Lengths of the 2 * pairs sequences, from half of the longest up."""
    most = case["longest"]
    return [max(1, most - (i * 37) % (most // 2 + 1)) for i in range(2 * case["pairs"])]


def _rows(case):
    return sum(_lengths(case)) + case["tail"] if case["op"] == "preference" else case["t"]


def _sizes(case):
    """Sizes of the tensors: three powers of ten, the total as given."""
    r = random.Random(case["total"] * 31 + case["count"])
    share = [10.0 ** r.uniform(-3.0, 0.0) for _ in range(case["count"])]
    got = [max(1, int((case["total"] - case["count"]) * s / sum(share))) for s in share]
    got[0] += case["total"] - sum(got)
    return got


def _prepare_adamw(case, g):
    sizes = _sizes(case)
    at, start = [], 0
    for n in sizes:  # each tensor starts at a whole block of one buffer
        at.append(start)
        start += -(-n // 128) * 128
    dev = "cuda"
    blocks = torch.tensor([-(-n // 128) for n in sizes], device=dev)
    ends = torch.tensor([a + n for a, n in zip(at, sizes)], device=dev).repeat_interleave(blocks)
    valid = torch.arange(start, device=dev).view(-1, 128) < ends[:, None]
    r = lambda: torch.randn((start // 128, 128), generator=g, device=dev) * valid
    level = torch.exp(1.5 * torch.randn((start // 128, 1), generator=g, device=dev))
    s = dict(case, sizes=sizes, p=(0.02 * r()).view(-1), t=STEP0)
    grad = 1e-4 * level * r()
    if case["grad"] == "fp8":
        amax = grad.abs().amax(1, keepdim=True)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        s["g"], s["g_scale"] = (grad / scale).to(torch.float8_e4m3fn).view(-1), scale.view(-1)
        s["grads"] = [(s["g"][a:a + n], s["g_scale"][a // 128:a // 128 - (-n // 128)]) for a, n in zip(at, sizes)]
    else:
        s["g"] = grad.view(-1).to(torch.float32 if case["grad"] == "f32" else torch.bfloat16)
        s["grads"] = [s["g"][a:a + n] for a, n in zip(at, sizes)]
    m, rt = 3e-5 * level * r(), 1e-4 * level * (0.3 + torch.rand(valid.shape, generator=g, device=dev)) * valid
    if case["bits"] == 8:
        for name, x in (("m", m), ("v", rt)):
            scale = x.abs().amax(1, keepdim=True).clamp(min=1e-30) / 448.0
            s[name], s[name + "_scale"] = (x / scale).to(torch.float8_e4m3fn).view(-1), scale.view(-1)
    else:
        s["m"], s["v"] = m.view(-1), rt.square().view(-1)
    s["copy"] = s["p"].bfloat16()
    s["decay"] = [0.1 if n >= 10000 else 0.0 for n in sizes]
    s["tensor"] = torch.arange(len(sizes), device=dev).repeat_interleave(blocks)[:, None]
    s["wd"] = torch.tensor(s["decay"], device=dev).repeat_interleave(blocks)[:, None]
    s["first"] = torch.tensor(at, device=dev).repeat_interleave(blocks)[:, None]
    s["seed"] = 12345
    s["max_norm"] = MAX_NORM if case["clip"] else None
    if own:
        from fp8_communication_compression_gb300 import AdamW

        part = lambda buf: [buf[a:a + n] for a, n in zip(at, sizes)]
        s["opt"] = AdamW(part(s["p"]), copies=part(s["copy"]), lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS,
                         weight_decay=s["decay"], state_bits=case["bits"], max_norm=s["max_norm"], seed=s["seed"])
        state = {"step": STEP0, "m": s["m"], "v": s["v"]}
        if case["bits"] == 8:
            state.update(m_scale=s["m_scale"], v_scale=s["v_scale"])
        s["opt"].load_state_dict(state)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "adamw":
        return _prepare_adamw(case, g)
    t, v, n = _rows(case), case["v"], case["n"]
    dt = torch.bfloat16 if case["dt"] == "bf16" else torch.float32
    rnd = lambda *sh: torch.randn(sh, generator=g, device="cuda")
    x = rnd(t, n).mul_(2.0)
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    x.scatter_add_(1, target[:, None], 4.0 + 3.0 * rnd(t, 1))
    s = dict(case, logits=x.to(dt), target=target)
    del x
    if case["op"] == "logprob":
        return s
    lse = torch.logsumexp(s["logits"][:, :v].double() / TAU, 1)
    if case["op"] == "logprob_grad":
        s["lse"], s["dlogp"] = lse.float(), rnd(t) / t
        return s
    logp = s["logits"].gather(1, target[:, None])[:, 0].double() / TAU - lse
    if case["op"] == "policy":
        # the first quarter of the rows is a prompt, which does not count
        keep = torch.arange(t, device="cuda") >= t // 4
        s["weight"] = keep.float() / (t - t // 4)
        # the policy has moved a little since; no ratio within 1e-3 of a border
        moved = 0.15 * rnd(t).double()
        for border in (math.log(1.0 - CLIP_LOW), math.log(1.0 + CLIP_HIGH)):
            moved = torch.where((moved - border).abs() < 1e-3, moved + 3e-3, moved)
        s["old"] = (logp - moved).float()
        s["advantage"] = rnd(t)
        s["ref"] = (logp + 0.2 * rnd(t).double()).float()
        return s
    lens = _lengths(case)
    s["offsets"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda")
    # each sequence begins with its prompt, and rows behind the last have no target
    lens_t = torch.tensor(lens, device="cuda")
    first = s["offsets"][:-1].repeat_interleave(lens_t)
    quarter = (lens_t // 4).repeat_interleave(lens_t)
    prompt = torch.arange(len(first), device="cuda") - first < quarter
    s["target"] = target.clone()
    s["target"][:len(first)][prompt] = -1
    s["target"][len(first):] = -1
    # the policy has moved from the reference by some nats in each sequence
    shift = (3.0 + 6.0 * torch.rand(len(lens), generator=g, device="cuda")) * (1.0 - 2.0 * (torch.arange(
        len(lens), device="cuda") % 2))
    if case["mean"]:
        shift = 0.3 * shift * lens_t
    s["ref"] = logp.float()
    s["ref"][:len(first)] -= (shift / (lens_t - lens_t // 4)).repeat_interleave(lens_t) + 0.02 * rnd(len(first))
    s["beta"] = 0.1
    return s


# -------------------------------------------------------------- plain form --

def _softmax(s):
    """x / tau, its maximum, the exponentials and their sum, in fp32."""
    x = s["logits"][:, :s["v"]].float() / TAU
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    return x, m, e, e.sum(1, keepdim=True)


def _plain_logp(s):
    x, m, e, z = _softmax(s)
    at = s["target"].clamp(min=0)[:, None]
    return (x.gather(1, at) - m - torch.log(z))[:, 0], e, z


def _plain_grad(s, coef, p):
    """coef / tau (1[target] - p) in the logits' type, p overwritten."""
    d = p.mul_(-(coef / TAU)[:, None])
    at = s["target"].clamp(min=0)[:, None]
    d.scatter_add_(1, at, (coef / TAU)[:, None])
    d = d.to(s["logits"].dtype)
    return torch.nn.functional.pad(d, (0, s["n"] - s["v"])) if s["n"] > s["v"] else d


def _plain_policy(s):
    logp, e, z = _plain_logp(s)
    w = s["weight"]
    r = torch.exp(logp - s["old"])
    free, held = r * s["advantage"], r.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * s["advantage"]
    d = s["ref"] - logp
    loss = w * (s["kl"] * (torch.expm1(d) - d) - torch.minimum(free, held))
    coef = w * (-s["kl"] * torch.expm1(d) - torch.where(free <= held, free, torch.zeros_like(free)))
    coef = torch.where(w != 0, coef, torch.zeros_like(coef))
    none = torch.zeros_like(logp)
    return {"loss": loss.double().sum().float(), "token_loss": torch.where(w != 0, loss, none),
            "logp": torch.where(w != 0, logp, none), "dlogits": _plain_grad(s, coef, e.div_(z))}


def _plain_preference(s):
    logp, e, z = _plain_logp(s)
    counts = s["target"] >= 0
    gap = torch.where(counts, logp.double() - s["ref"], torch.zeros_like(logp, dtype=torch.float64))
    total = torch.nn.functional.pad(gap.cumsum(0), (1, 0))
    ratio = total[s["offsets"][1:]] - total[s["offsets"][:-1]]
    tokens = torch.nn.functional.pad(counts.long().cumsum(0), (1, 0))
    tokens = (tokens[s["offsets"][1:]] - tokens[s["offsets"][:-1]]).clamp(min=1)
    if s["mean"]:
        ratio = ratio / tokens
    margin = s["beta"] * (ratio[0::2] - ratio[1::2])
    ls = s["ls"]
    loss = (1.0 - ls) * torch.log1p(torch.exp(-margin)) + ls * torch.log1p(torch.exp(margin))
    slope = (ls - 1.0 / (1.0 + torch.exp(margin))) * s["beta"] / len(margin)
    slope = torch.stack((slope, -slope), 1).view(-1)
    if s["mean"]:
        slope = slope / tokens
    lens = s["offsets"].diff()
    coef = torch.zeros_like(logp)
    coef[:int(sum(_lengths(s)))] = slope.float().repeat_interleave(lens)
    coef = torch.where(counts, coef, torch.zeros_like(coef))
    return {"loss": loss.mean().float(), "margin": margin.float(), "logratio": ratio.float(),
            "logp": torch.where(counts, logp, torch.zeros_like(logp)), "dlogits": _plain_grad(s, coef, e.div_(z))}


MASK32 = (1 << 32) - 1


def _mix(x):
    """Hash of a 32-bit whole number (held in 64 bits), to 32 bits."""
    x = ((x ^ (x >> 16)) * 0x9E3779B1) & MASK32
    x = ((x ^ (x >> 15)) * 0x85A308D3) & MASK32
    return x ^ (x >> 16)


def _random32(s):
    """32 random bits for each element of the step that is being done."""
    dev = s["p"].device
    at = torch.arange(s["p"].numel(), device=dev).view(-1, 128) - s["first"]
    key = _mix(torch.tensor(s["seed"] & MASK32, device=dev))
    key = _mix(key ^ ((s["seed"] >> 32) & MASK32))
    key = _mix(key ^ (s["t"] & MASK32))
    key = _mix(key ^ s["tensor"])
    return _mix(((at * 0x13198A2F) & MASK32) ^ key)  # tensors here have less than 2^32 elements


def _store8(x, bits, least):
    """E4M3 values and multipliers of blocks of x, rounded up with the
    probability of the rest: bits (0 .. 65535) and a half of 65536."""
    amax = x.abs().amax(1, keepdim=True)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    y = (x.abs() * torch.where(amax > 0, 448.0 / amax, torch.ones_like(amax))).clamp(max=448.0)
    # below 2^-6 the steps are those of 2^-6
    low = y < 2.0 ** -6
    f = torch.where(low, y + 2.0 ** -6, y).contiguous().view(torch.int32)
    f = ((f + (bits << 4) + 8) >> 20 << 20).to(torch.int32).view(torch.float32)
    q = torch.where(low, f - 2.0 ** -6, f)
    if least:
        q = torch.where((x > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    return torch.copysign(q, x).to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def _plain_adamw(s):
    blocks = (-1, 128)
    g = s["g"].float().view(blocks)
    if s["grad"] == "fp8":
        g = g * s["g_scale"][:, None]
    out, coef = {}, None
    if s["max_norm"] is not None:
        norm = g.square().sum(1).double().sum().sqrt().float()
        out["norm"] = norm
        coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        g = g * coef
    if s["bits"] == 8:
        bits = _random32(s)
        m = s["m"].float().view(blocks) * s["m_scale"][:, None]
        v = (s["v"].float().view(blocks) * s["v_scale"][:, None]).square()
    else:
        m, v = s["m"].view(blocks), s["v"].view(blocks)
    s["t"] += 1
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g * g
    root = torch.sqrt(v)
    p = s["p"].view(blocks)
    step = (m / (1.0 - BETA1 ** s["t"])) / (root / math.sqrt(1.0 - BETA2 ** s["t"]) + ADAM_EPS)
    s["p"] = (p - LR * (s["wd"] * p + step)).view(-1)
    s["copy"] = s["p"].bfloat16()
    if s["bits"] == 8:
        s["m"], s["m_scale"] = _store8(m, (bits & 0xFFFF).int(), False)
        s["v"], s["v_scale"] = _store8(root, (bits >> 16).int(), True)
        out |= {"m_scale": s["m_scale"], "v_scale": s["v_scale"]}
    else:
        s["m"], s["v"] = m.view(-1), v.view(-1)
    return out | {"p": s["p"], "copy": s["copy"], "m": s["m"], "v": s["v"]}


def _plain(s):
    op = s["op"]
    if op == "logprob":
        x, m, e, z = _softmax(s)
        at = x.gather(1, s["target"][:, None])
        return {"logp": (at - m - torch.log(z))[:, 0], "lse": (m + torch.log(z))[:, 0]}
    if op == "logprob_grad":
        p = torch.exp(s["logits"][:, :s["v"]].float() / TAU - s["lse"][:, None])
        return _plain_grad(s, s["dlogp"], p)
    return _plain_policy(s) if op == "policy" else _plain_preference(s) if op == "preference" else _plain_adamw(s)


def run(s):
    if not own:
        return _plain(s)
    from fp8_communication_compression_gb300 import api

    op = s["op"]
    if op == "logprob":
        logp, lse = api.token_logprob(s["logits"], s["target"], vocab=s["v"], temperature=TAU)
        return {"logp": logp, "lse": lse}
    if op == "logprob_grad":
        return api.token_logprob_backward(s["dlogp"], s["logits"], s["target"], s["lse"], vocab=s["v"],
                                          temperature=TAU)
    if op == "policy":
        got = api.policy_loss(s["logits"], s["target"], s["old"], s["advantage"], s["weight"],
                              ref_logp=s["ref"] if s["kl"] else None, clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                              kl=s["kl"], vocab=s["v"], temperature=TAU)
        return {"loss": got.loss, "token_loss": got.token_loss, "logp": got.logp, "dlogits": got.dlogits}
    if op == "preference":
        got = api.preference_loss(s["logits"], s["target"], s["offsets"], s["ref"], beta=s["beta"],
                                  label_smoothing=s["ls"], mean=s["mean"], vocab=s["v"], temperature=TAU)
        return {"loss": got.loss, "margin": got.margin, "logratio": got.logratio, "logp": got.logp,
                "dlogits": got.dlogits}
    opt = s["opt"]
    norm = opt.step(s["grads"])
    out = {"p": s["p"], "copy": s["copy"], "m": opt.m, "v": opt.v}
    if norm is not None:
        out["norm"] = norm
    if s["bits"] == 8:
        out |= {"m_scale": opt.m_scale, "v_scale": opt.v_scale}
    return out


def work(case):
    if case["op"] == "adamw":
        n, blocks = case["total"], sum(-(-k // 128) for k in _sizes(case))
        grad = {"f32": 4 * n, "bf16": 2 * n, "fp8": n + 4 * blocks}[case["grad"]]
        state = 16 * n if case["bits"] == 32 else 4 * n + 16 * blocks
        # the weights read and written, their bf16 copy written
        return {"bytes": 10 * n + grad + state, "flops": (60 if case["bits"] == 8 else 15) * n}
    t, v, n, e = _rows(case), case["v"], case["n"], 2 if case["dt"] == "bf16" else 4
    if case["op"] == "logprob":
        return {"bytes": t * v * e + 16 * t, "flops": 4 * t * v}
    if case["op"] == "logprob_grad":
        return {"bytes": t * (v + n) * e + 16 * t, "flops": 4 * t * v}
    rows = t - t // 4 if case["op"] == "policy" else sum(k - k // 4 for k in _lengths(case))
    return {"bytes": (rows * v + t * n) * e + 32 * t, "flops": 8 * rows * v}


# ------------------------------------------------------- values in 64 bits --

def _exact_adamw(case, seed):
    s = prepare(case, seed)
    d = lambda name: s[name].double().view(-1, 128)
    g = d("g") * s["g_scale"].double()[:, None] if case["grad"] == "fp8" else d("g")
    out = {}
    if case["clip"]:
        out["norm"] = torch.linalg.vector_norm(g)
        g = g * min(1.0, MAX_NORM / (float(out["norm"]) + 1e-6))
    m, v = d("m"), d("v")
    if case["bits"] == 8:
        m, v = m * s["m_scale"].double()[:, None], (v * s["v_scale"].double()[:, None]) ** 2
    m = m + (1.0 - BETA1) * (g - m)
    v = v + (1.0 - BETA2) * (g * g - v)
    t = STEP0 + 1
    p = d("p") * (1.0 - LR * s["wd"].double())
    p = p - LR * m / (1.0 - BETA1 ** t) / ((v / (1.0 - BETA2 ** t)) ** 0.5 + ADAM_EPS)
    out |= {"p": p.view(-1), "copy": p.view(-1), "m": m.view(-1), "v": v.view(-1)}
    if case["bits"] == 32:
        return out

    def h(x):  # the hash by division and remainders of whole numbers
        for shift, factor in ((16, 0x9E3779B1), (15, 0x85A308D3)):
            x = (x ^ (x // (1 << shift))) * factor % (1 << 32)
        return x ^ (x // (1 << 16))

    key = h(h(h(s["seed"] % (1 << 32)) ^ (s["seed"] >> 32)) ^ STEP0)
    key = torch.tensor([h(key ^ i) for i in range(case["count"])], device=m.device)[s["tensor"]]
    at = torch.arange(m.numel(), device=m.device).view(-1, 128) - s["first"]
    x = (at * 0x13198A2F) % (1 << 32) ^ key
    x = (x ^ (x >> 16)) * 0x9E3779B1 % (1 << 32)
    x = (x ^ (x >> 15)) * 0x85A308D3 % (1 << 32)
    x = x ^ (x >> 16)
    for name, value, u in (("m", m, x % 65536), ("v", v.sqrt(), x // 65536)):
        top = value.abs().amax(1, keepdim=True)
        scale = torch.where(top > 0, top / 448.0, 1.0)
        y = value.abs() / scale
        _, e = torch.frexp(y)
        step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
        q = torch.floor(y / step + (u.double() + 0.5) / 65536.0) * step
        q = torch.where(y >= 448.0 * (1.0 - 1e-12), 448.0, q)
        if name == "v":
            q = torch.where((value > 0) & (q == 0), 2.0 ** -9, q)
        out[name], out[name + "_scale"] = (q * value.sign()).view(-1), scale.view(-1)
    return out


def exact(case, seed):
    if case["op"] == "adamw":
        return _exact_adamw(case, seed)
    s = prepare(case, seed)
    op, v = case["op"], case["v"]
    if op == "logprob_grad":
        q = s["logits"].double() / TAU - s["lse"].double()[:, None]
        grad = -q.exp() * s["dlogp"].double()[:, None] / TAU
        grad[:, v:] = 0.0
        rows = torch.arange(case["t"], device=q.device)
        grad[rows, s["target"]] += s["dlogp"].double() / TAU
        return grad
    # the gradients by reverse differentiation of the definitions in float64
    x = s["logits"].double()
    if op != "logprob":
        x.requires_grad_()
    rows = torch.arange(x.shape[0], device=x.device)
    lse = torch.logsumexp(x[:, :v] / TAU, 1)
    logp = x[rows, s["target"].clamp(min=0)] / TAU - lse
    if op == "logprob":
        return {"logp": logp, "lse": lse}
    if op == "policy":
        keep = s["weight"] > 0
        ratio = (logp - s["old"].double()).exp()
        a = s["advantage"].double()
        gain = torch.where(a > 0, torch.where(ratio > 1.0 + CLIP_HIGH, (1.0 + CLIP_HIGH) * a, ratio * a),
                           torch.where(ratio < 1.0 - CLIP_LOW, (1.0 - CLIP_LOW) * a, ratio * a))
        gap = s["ref"].double() - logp
        per = s["weight"].double() * (case["kl"] * (gap.exp() - gap - 1.0) - gain)
        loss = per[keep].sum()
        (grad,) = torch.autograd.grad(loss, x)
        return {"loss": loss.detach(), "token_loss": (per * keep).detach(), "logp": (logp * keep).detach(),
                "dlogits": grad}
    counts = s["target"] >= 0
    gap = (logp - s["ref"].double()) * counts
    sums = [gap[a:b].sum() / (max(1, int(counts[a:b].sum())) if case["mean"] else 1)
            for a, b in zip(s["offsets"].tolist(), s["offsets"].tolist()[1:])]
    ratio = torch.stack(sums)
    z = s["beta"] * (ratio[0::2] - ratio[1::2])
    loss = -((1.0 - case["ls"]) * torch.log(torch.sigmoid(z)) + case["ls"] * torch.log(torch.sigmoid(-z))).mean()
    (grad,) = torch.autograd.grad(loss, x)
    return {"loss": loss.detach(), "margin": z.detach(), "logratio": ratio.detach(),
            "logp": (logp * counts).detach(), "dlogits": grad}
