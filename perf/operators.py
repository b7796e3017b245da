"""Cases, plain forms and 64-bit values of the FP8 linear layer and of the
norms around a block.

Operators (``case["op"]``):

* ``linear``: y = Q(x) Qw^T, the activation quantised in the call (E4M3, one
  power-of-two scale per 128 values of a row), the weight held quantised (one
  scale per 128 x 128 tile).
* ``linear_grad``: its backward pass, dx = Q(dy) Qw and dw = Qc(dy)^T Qc(x),
  Qc quantising in blocks of 128 tokens.
* ``norm``: z = rmsnorm(y) g_post, h' = s h + gate z, n = rmsnorm(h') g_pre.
* ``norm_grad``: its backward pass.
* ``norm_linear``: the same norms with n quantised as it is written, and the
  product that reads it.

The scale of a block is 2^E with the smallest E such that amax <= 448 2^E
(and E >= -127; E = 0 for a block of zeros).
"""

import math

import torch

own = False

GATES = ("none", "channel", "token", "full")


def listed():
    return [
        # one token through a GPT-6.7B-sized projection: latency and the weight's bytes
        {"name": "linear_1_4096_4096", "op": "linear", "m": 1, "k": 4096, "n": 4096},
        # a few tokens through the GPT-2.7B up-projection
        {"name": "linear_37_2560_10240", "op": "linear", "m": 37, "k": 2560, "n": 10240},
        # a ragged batch with sizes that fill no tile
        {"name": "linear_777_1300_5119", "op": "linear", "m": 777, "k": 1300, "n": 5119},
        # the GPT-6.7B row-parallel projection of a training step
        {"name": "linear_8192_4096_4096", "op": "linear", "m": 8192, "k": 4096, "n": 4096},
        # odd sizes backward
        {"name": "linear_grad_513_1000_777", "op": "linear_grad", "m": 513, "k": 1000, "n": 777},
        # GPT-2.7B up-projection backward
        {"name": "linear_grad_4096_2560_10240", "op": "linear_grad", "m": 4096, "k": 2560, "n": 10240},
        # GPT-6.7B up-projection backward, the largest
        {"name": "linear_grad_8192_4096_16384", "op": "linear_grad", "m": 8192, "k": 4096, "n": 16384},
        # a single token's norms
        {"name": "norm_1_4096_channel", "op": "norm", "t": 1, "d": 4096, "gate": "channel", "s": 1.0},
        # GPT-13B rows, a gate computed from the tokens
        {"name": "norm_8192_5120_full", "op": "norm", "t": 8192, "d": 5120, "gate": "full", "s": 0.5},
        # GPT-6.7B rows backward, a learned gate
        {"name": "norm_grad_8192_4096_channel", "op": "norm_grad", "t": 8192, "d": 4096, "gate": "channel", "s": 1.0},
        # an odd width backward, one gate value a token
        {"name": "norm_grad_515_2561_token", "op": "norm_grad", "t": 515, "d": 2561, "gate": "token", "s": 0.7},
        # the norms writing the up-projection's FP8 operand, GPT-2.7B
        {"name": "norm_linear_4096_2560_10240", "op": "norm_linear", "t": 4096, "d": 2560, "n": 10240,
         "gate": "none", "s": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A width: most are multiples of 16, some are odd."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.3 else max(16, v // 16 * 16)


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_grad", "norm", "norm_grad", "norm_linear"))
    if op in ("linear", "linear_grad"):
        return {"op": op, "m": _log(rng, 1, 8192), "k": _size(rng, 128, 4096), "n": _size(rng, 128, 16384)}
    case = {"op": op, "t": _log(rng, 1, 8192), "d": _size(rng, 128, 5120), "gate": rng.choice(GATES),
            "s": rng.choice((1.0, 0.5, 0.7))}
    if op == "norm_linear":
        case["n"] = _size(rng, 128, 10240)
    return case


# ------------------------------------------------------------------ inputs --

def _activation(g, rows, cols):
    """Near-zero-dense and long-tailed values with channel scales, bf16."""
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    u = torch.rand((rows, cols), generator=g, device="cuda")
    x = r(rows, cols)
    x = torch.where(u < 0.9, 0.05 * x, x)
    x = torch.where(u > 0.999, 6.0 * x, x)
    return (x * torch.exp(-2.0 * torch.rand((1, cols), generator=g, device="cuda"))).bfloat16()


def _up(v, m):
    return -(-v // m) * m


def _weight(g, n, k):
    """A weight as a program keeps it: E4M3 codes [n, k to 16], a scale byte
    per 128 x 128 tile, and both transposed."""
    w = 0.02 * torch.randn((n, k), generator=g, device="cuda")
    kb, nb = _up(k, 128) // 128, _up(n, 128) // 128
    t = torch.zeros((nb * 128, kb * 128), device="cuda")
    t[:n, :k] = w
    t = t.view(nb, 128, kb, 128)
    byte = _scale_byte(t.abs().amax(dim=(1, 3)))
    q = (t * _inverse_scale(byte)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    q = q.view(nb * 128, kb * 128)
    byte = byte.to(torch.uint8)
    return {"codes": q[:n, :_up(k, 16)].contiguous(), "scale": byte.t().contiguous(),
            "codes_t": q.t()[:k, :_up(n, 16)].contiguous(), "scale_t": byte.contiguous()}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] in ("linear", "linear_grad"):
        s["x"] = _activation(g, case["m"], case["k"])
        s["w"] = _weight(g, case["n"], case["k"])
        if case["op"] == "linear_grad":
            s["dy"] = (1e-3 * _activation(g, case["m"], case["n"]).float()).bfloat16()
        return s
    t, d = case["t"], case["d"]
    r = lambda *sh: torch.randn(sh, generator=g, device="cuda")
    s["y"] = _activation(g, t, d)
    s["h"] = (2.0 * r(t, d)).bfloat16()
    s["g_post"] = 1.0 + 0.1 * r(d)
    s["g_pre"] = 1.0 + 0.1 * r(d)
    s["gv"] = {"none": None, "channel": 0.5 + 0.1 * r(d), "token": torch.sigmoid(r(t, 1)),
               "full": torch.sigmoid(r(t, d)).bfloat16()}[case["gate"]]
    if case["op"] == "norm_grad":
        s["dn"] = (1e-2 * r(t, d)).bfloat16()
        s["dh"] = (1e-2 * r(t, d)).bfloat16()
    if case["op"] == "norm_linear":
        s["w"] = _weight(g, case["n"], d)
    return s


# -------------------------------------------------------------- plain form --

EPS = 1e-6


def _scale_byte(amax):
    """E + 127 for the smallest E with amax <= 448 2^E, as int32: 448 is
    1.75 2^8, so E is amax's exponent - 8, one more above 1.75."""
    b = amax.contiguous().view(torch.int32)
    return torch.where(b == 0, 127, (((b + 0x1FFFFF) >> 23) - 8).clamp(min=0))


def _scale(byte):
    """2^(byte - 127) in fp32 from its bits, exactly (exp2 may be an ulp off)."""
    n = (byte.clamp(min=1) << 23).view(torch.float32)
    return torch.where(byte == 0, 2.0 ** -127, n)


def _inverse_scale(byte):
    """2^(127 - byte), likewise; the product with a value is then exact, so
    the ties of the rounding to E4M3 are the value's own."""
    return ((254 - byte) << 23).view(torch.float32)


def _quantised(x):
    """[rows, c] -> the fp32 values its codes and scales stand for."""
    rows, c = x.shape
    t = torch.nn.functional.pad(x.float(), (0, _up(c, 128) - c)).view(rows, -1, 128)
    byte = _scale_byte(t.abs().amax(dim=2, keepdim=True))
    q = (t * _inverse_scale(byte)).to(torch.float8_e4m3fn).float() * _scale(byte)
    return q.view(rows, -1)[:, :c]


def _weight_values(codes, scale, n, k):
    v = codes.view(torch.float8_e4m3fn).float()
    sc = _scale(scale.to(torch.int32)).t().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    return v[:, :k] * sc[:, :k]


def _norms(s):
    y, h = s["y"].float(), s["h"].float()
    z = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * s["g_post"]
    if s["gv"] is not None:
        z = z * s["gv"].float()
    h2 = s["s"] * h + z
    return h2, h2 * torch.rsqrt(h2.square().mean(1, keepdim=True) + EPS) * s["g_pre"]


def _norms_grad(s):
    # s["h"] is the residual stream after the block
    y, h2, dn = s["y"].float(), s["h"].float(), s["dn"].float()
    ry = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    rh = torch.rsqrt(h2.square().mean(1, keepdim=True) + EPS)
    u = dn * s["g_pre"]
    g = s["dh"].float() + rh * (u - h2 * rh.square() * (u * h2).mean(1, keepdim=True))
    gate = 1.0 if s["gv"] is None else s["gv"].float()
    z = y * ry * s["g_post"]
    dz = g * gate
    v = dz * s["g_post"]
    dy = ry * (v - y * ry.square() * (v * y).mean(1, keepdim=True))
    out = {"dy": dy.bfloat16(), "dh": (s["s"] * g).bfloat16(), "dg_pre": (dn * h2 * rh).sum(0),
           "dg_post": (dz * y * ry).sum(0)}
    if s["gate"] == "channel":
        out["dgate"] = (g * z).sum(0)
    elif s["gate"] == "token":
        out["dgate"] = (g * z).sum(1, keepdim=True)
    elif s["gate"] == "full":
        out["dgate"] = (g * z).bfloat16()
    return out


def _plain(s):
    op = s["op"]
    if op == "linear":
        w = _weight_values(s["w"]["codes"], s["w"]["scale"], s["n"], s["k"])
        return (_quantised(s["x"]) @ w.t()).bfloat16()
    if op == "linear_grad":
        w = _weight_values(s["w"]["codes"], s["w"]["scale"], s["n"], s["k"])
        dx = (_quantised(s["dy"]) @ w).bfloat16()
        dw = _quantised(s["dy"].t()) @ _quantised(s["x"].t()).t()
        return {"dx": dx, "dw": dw}
    if op == "norm":
        h2, n = _norms(s)
        return {"h": h2.bfloat16(), "n": n.bfloat16()}
    if op == "norm_grad":
        return _norms_grad(s)
    h2, n = _norms(s)
    w = _weight_values(s["w"]["codes"], s["w"]["scale"], s["n"], s["d"])
    return {"h": h2.bfloat16(), "y": (_quantised(n) @ w.t()).bfloat16()}


def run(s):
    if not own:
        return _plain(s)
    from fp8_communication_compression_gb300 import api

    op = s["op"]
    if op == "linear":
        return api.fp8_linear(s["x"], s["w"]["codes"], s["w"]["scale"])
    if op == "linear_grad":
        dx, dw = api.fp8_linear_backward(s["dy"], s["x"], s["w"]["codes_t"], s["w"]["scale_t"])
        return {"dx": dx, "dw": dw}
    if op == "norm":
        h2, n = api.rmsnorm_gate_residual(s["y"], s["h"], s["g_post"], s["g_pre"], s["gv"], s["s"], EPS)
        return {"h": h2, "n": n}
    if op == "norm_grad":
        dy, dh, dg_post, dg_pre, dgate = api.rmsnorm_gate_residual_backward(
            s["dn"], s["dh"], s["y"], s["h"], s["g_post"], s["g_pre"], s["gv"], s["s"], EPS)
        out = {"dy": dy, "dh": dh, "dg_pre": dg_pre, "dg_post": dg_post}
        if dgate is not None:
            out["dgate"] = dgate
        return out
    h2, codes, scale = api.rmsnorm_gate_residual_fp8(s["y"], s["h"], s["g_post"], s["g_pre"], s["gv"], s["s"], EPS)
    return {"h": h2, "y": api.fp8_gemm(codes, scale, s["w"]["codes"], s["w"]["scale"])}


def work(case):
    op = case["op"]
    gate = {"none": lambda t, d: 0, "channel": lambda t, d: 4 * d, "token": lambda t, d: 4 * t,
            "full": lambda t, d: 2 * t * d}
    blocks = lambda r, c: (_up(r, 128) // 128) * (_up(c, 128) // 128)
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * m * k + n * k + blocks(n, k) + 2 * m * n, "flops": 2 * m * n * k}
    if op == "linear_grad":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * m * n + 2 * m * k + n * k + blocks(n, k) + 2 * m * k + 4 * n * k, "flops": 4 * m * n * k}
    t, d = case["t"], case["d"]
    gb = gate[case["gate"]](t, d)
    if op == "norm":
        return {"bytes": 8 * t * d + 8 * d + gb, "flops": 12 * t * d}
    if op == "norm_grad":
        return {"bytes": 12 * t * d + 16 * d + 2 * gb, "flops": 30 * t * d}
    n = case["n"]
    return {"bytes": 6 * t * d + 8 * d + gb + n * d + blocks(n, d) + 2 * t * n, "flops": 2 * t * d * n + 12 * t * d}


# ------------------------------------------------------- values in 64 bits --

def _power(e):
    """2^e in float64 from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _q64(x):
    """Quantised values of float64 rows, from the definition: 2^E by frexp
    (amax = f 2^e, f in [0.5, 1): amax <= 448 2^E = 0.875 2^(E + 9)), then
    the nearest multiple of E4M3's step at each value, ties to even."""
    rows, c = x.shape
    pad = torch.zeros((rows, _up(c, 128)), dtype=torch.float64, device=x.device)
    pad[:, :c] = x
    b = pad.reshape(rows, -1, 128)
    f, e = torch.frexp(b.abs().amax(dim=2, keepdim=True))
    e = torch.where(f <= 0.875, e - 9, e - 8).clamp(min=-127)
    v = b * _power(-e)
    _, ev = torch.frexp(v)
    step = _power((ev - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step * _power(e)).reshape(rows, -1)[:, :c]


def _w64(w, n, k):
    """The weight's values from its codes' bits."""
    c = w["codes"][:, :k].long()
    ex, mant = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ex == 0, mant * 2.0 ** -9, (1.0 + mant / 8.0) * _power(ex - 7))
    v = torch.where(c >= 128, -mag, mag)
    i = torch.arange(n, device=c.device) // 128
    j = torch.arange(k, device=c.device) // 128
    return v * _power(w["scale"].long() - 127)[j][:, i].t()


def _norms64(s):
    y, h = s["y"].double(), s["h"].double()
    gate = 1.0 if s["gv"] is None else s["gv"].double()
    yn = y / ((y * y).sum(1, keepdim=True) / y.shape[1] + EPS).sqrt()
    h2 = s["s"] * h + gate * (yn * s["g_post"].double())
    return h2, h2 / ((h2 * h2).sum(1, keepdim=True) / h2.shape[1] + EPS).sqrt() * s["g_pre"].double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _q64(s["x"].double()) @ _w64(s["w"], case["n"], case["k"]).t()
    if op == "linear_grad":
        dy, x = s["dy"].double(), s["x"].double()
        dx = _q64(dy) @ _w64(s["w"], case["n"], case["k"])
        return {"dx": dx, "dw": _q64(dy.t().contiguous()) @ _q64(x.t().contiguous()).t()}
    if op == "norm":
        h2, n = _norms64(s)
        return {"h": h2, "n": n}
    if op == "norm_linear":
        h2, n = _norms64(s)
        return {"h": h2, "y": _q64(n) @ _w64(s["w"], case["n"], case["d"]).t()}
    # the gradient by reverse differentiation of the definition in float64
    y = s["y"].double().requires_grad_()
    gp, gq = s["g_post"].double().requires_grad_(), s["g_pre"].double().requires_grad_()
    gate = None if s["gv"] is None else s["gv"].double().requires_grad_()
    h2 = s["h"].double()
    # h' is given: the forward's h' = s h + gate z is linear in h, so take
    # z's part as y moves and h as what is left
    z = y / (y.square().mean(1, keepdim=True) + EPS).sqrt() * gp
    gz = z if gate is None else z * gate
    h = ((h2 - gz.detach()) / case["s"]).requires_grad_()
    h2 = case["s"] * h + gz
    n = h2 / (h2.square().mean(1, keepdim=True) + EPS).sqrt() * gq
    loss = (n * s["dn"].double()).sum() + (h2 * s["dh"].double()).sum()
    wrt = [y, h, gq, gp] + ([] if gate is None else [gate])
    got = torch.autograd.grad(loss, wrt)
    out = {"dy": got[0], "dh": got[1], "dg_pre": got[2], "dg_post": got[3]}
    if gate is not None:
        out["dgate"] = got[4]
    return out
