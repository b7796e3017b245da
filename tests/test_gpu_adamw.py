"""grad_norm and AdamW on the GPU against the float64 forms, whose bounds
training_reference.py derives.  A code of the 8-bit states may be any that a
value within its bound is held as under the given random bits."""

import math

import numpy as np
import pytest
import torch

import fp8_reference as F
import training_reference as R
from fp8_communication_compression_gb300 import AdamW, _lib, api

pytestmark = pytest.mark.gpu

BETAS, EPS = (0.9, 0.95), 1e-8


def main_gradient(g):
    """A gradient as an FP8 main gradient (codes, multipliers), and its values."""
    b = R.pad(g)
    amax = b.abs().amax(1, keepdim=True)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = (b / scale).to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[:g.numel()]
    return codes.cuda(), scale.view(-1).cuda()


def values(g):
    """float64 values of a gradient as it is given to the calls."""
    if isinstance(g, tuple):
        n = g[0].numel()
        return (R.pad(F.code_values(g[0])) * g[1].cpu().double()[:, None]).view(-1)[:n]
    return g.cpu().double().reshape(-1)


def gradients(sizes, kinds, gen, level=1e-3):
    out = []
    for i, n in enumerate(sizes):
        g = level * torch.randn(n, generator=gen) * math.exp(float(torch.randn(1, generator=gen)))
        kind = kinds[i % len(kinds)]
        out.append(main_gradient(g) if kind == "fp8" else g.to(torch.bfloat16 if kind == "bf16" else torch.float32).cuda())
    return out


SIZES = [[1], [3, 0, 128], [127, 129, 4096, 5], [1000003], [4097] * 17, [33 + 7 * i for i in range(400)],
         [5 + i for i in range(1000)]]
KINDS = [("f32",), ("bf16",), ("fp8",), ("fp8", "f32", "bf16")]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("kinds", KINDS, ids="-".join)
def test_grad_norm(sizes, kinds):
    grads = gradients(sizes, kinds, torch.Generator().manual_seed(1))
    want = math.sqrt(sum(float(values(g).square().sum()) for g in grads))
    got = api.grad_norm(grads, 0.5)
    # squares and short sums in fp32 (32 terms in a row at most), the rest in fp64
    assert got.shape == () and abs(float(got) - 0.5 * want) <= 40 * R.U * want
    assert torch.equal(got, api.grad_norm(grads, -0.5))


def test_grad_norm_of_values_that_are_not_finite():
    g = torch.zeros(1000, device="cuda")
    assert float(api.grad_norm([g])) == 0.0
    for bad in (math.inf, -math.inf, math.nan, 1e30):
        g[777] = bad
        assert not api.grad_norm([torch.zeros(5, device="cuda"), g]).isfinite()


def states(opt, seed, level=1e-3):
    """A state as of a step later than the first."""
    gen = torch.Generator().manual_seed(seed)
    d = {"step": 41}
    n = opt.m.numel()
    m, r = level * torch.randn(n, generator=gen), level * (0.1 + torch.rand(n, generator=gen))
    mask = torch.zeros(n, dtype=torch.bool)
    for a, k in zip(opt.starts, opt.sizes):
        mask[a:a + k] = True
    m, r = m * mask, r * mask
    if opt.state_bits == 32:
        return d | {"m": m.cuda(), "v": r.square().cuda()}
    for name, x in (("m", m), ("v", r)):
        codes, scale = main_gradient(x)
        d[name], d[name + "_scale"] = codes.view(torch.float8_e4m3fn), scale
    return d


def state_values(opt, i):
    """(m, v) of tensor i in float64."""
    a, n = opt.starts[i], opt.sizes[i]
    if opt.state_bits == 32:
        return opt.m[a:a + n].cpu().double(), opt.v[a:a + n].cpu().double()
    got = []
    for c, s in ((opt.m, opt.m_scale), (opt.v, opt.v_scale)):
        sc = s[a // 128:a // 128 - (-n // 128)].cpu().double()
        got.append((R.pad(F.code_values(c[a:a + n].view(torch.uint8))) * sc[:, None]).view(-1)[:n])
    return got[0], got[1].square()


def check_step(opt, grads, before, lr, wd, t, coef, tol_coef, scale=1.0):
    for i, g in enumerate(grads):
        n = opt.sizes[i]
        if n == 0:
            continue
        p0, m0, v0 = before[i]
        (p, dp), (m, dm), (v, dv), (r, dr) = R.adamw(p0, values(g), m0, v0, t, lr[i], wd[i], *BETAS, EPS, coef, tol_coef)
        got = opt.params[i].cpu().double().view(-1)
        assert ((got - p).abs() <= dp).all(), (i, float(((got - p).abs() - dp).max()))
        if opt.copies[i] is not None:
            assert torch.equal(opt.copies[i], opt.params[i].bfloat16())
        a = opt.starts[i]
        if opt.state_bits == 32:
            assert ((opt.m[a:a + n].cpu().double() - m).abs() <= dm).all()
            assert ((opt.v[a:a + n].cpu().double() - v).abs() <= dv).all()
            continue
        bits = R.bits_of(n, i, t - 1, opt.seed)
        for codes, scales, x, dx, u, least in ((opt.m, opt.m_scale, m, dm, bits & 0xFFFF, False),
                                               (opt.v, opt.v_scale, r, dr, bits >> 16, True)):
            lo, hi, sc, dsc = R.code_range(x, dx, u, least)
            q = F.code_values(codes[a:a + n].view(torch.uint8))
            assert ((lo <= q.abs()) & (q.abs() <= hi)).all()
            assert float((lo == hi).double().mean()) > 0.99 or n < 1000   # the bound says something
            assert ((q == 0) | (torch.sign(q) == torch.sign(x)) | (x.abs() <= dx)).all()
            assert ((scales[a // 128:a // 128 - (-n // 128)].cpu().double() - sc).abs() <= dsc).all()
        pad = codes[a + n:a - (-n // 128) * 128].view(torch.uint8)
        assert not pad.any()


# large sizes are clipped with mixed gradients only
STEPS = [(s, k, b, c) for c in (None, 0.01) for b in (8, 32) for k in KINDS for s in SIZES
         if not (c and sum(s) > 100000 and len(k) == 1)]


@pytest.mark.parametrize("sizes,kinds,bits,clip", STEPS,
                         ids=[f"{len(s)}x{s[0]}-{'-'.join(k)}-{b}-{c}" for s, k, b, c in STEPS])
def test_steps(sizes, kinds, bits, clip):
    gen = torch.Generator().manual_seed(2)
    params = [(0.05 * torch.randn(n, generator=gen)).cuda() for n in sizes]
    copies = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") if i % 3 != 1 else None for i, n in enumerate(sizes)]
    lr = [1e-3 * (1 + i % 4) for i in range(len(sizes))]
    wd = [0.1 * (i % 2) for i in range(len(sizes))]
    opt = AdamW(params, copies, lr, BETAS, EPS, wd, bits, clip, seed=(7 << 32) + 9)
    opt.load_state_dict(states(opt, 3))
    factor = torch.tensor([0.5], device="cuda")
    for k in range(2):
        before = [(p.cpu().double().view(-1), *state_values(opt, i)) for i, p in enumerate(params)]
        grads = gradients(sizes, kinds, gen)
        norm = opt.step(grads, grad_scale=0.25, lr_factor=factor)
        coef, tol = 0.25, 0.0
        if clip:
            want = 0.25 * math.sqrt(sum(float(values(g).square().sum()) for g in grads))
            assert abs(float(norm) - want) <= 40 * R.U * want
            coef, tol = 0.25 * min(1.0, clip / (want + 1e-6)), 46 * R.U
        else:
            assert norm is None
        assert opt.steps.tolist() == [42 + k, 0]
        # lr and weight decay reach the kernel as fp32
        f = lambda v: float(np.float32(v))
        check_step(opt, grads, before, [f(v) * 0.5 for v in lr], [f(v) for v in wd], 42 + k, coef, tol)


def test_first_step_from_nothing():
    for bits in (8, 32):
        p = torch.ones(300, device="cuda")
        opt = AdamW([p], lr=0.1, state_bits=bits)
        g = torch.full((300,), 2.0, device="cuda")
        g[5] = 0.0
        opt.step([g])
        # m / (1 - b1) = g and sqrt(v / (1 - b2)) = |g|: a whole step of lr
        want = torch.full((300,), 0.9)
        want[5] = 1.0
        assert torch.allclose(p.cpu(), want, rtol=0, atol=1e-6)


def test_a_step_that_is_not_finite_is_left_out():
    for bits in (8, 32):
        p, c = torch.randn(1000, device="cuda"), torch.zeros(1000, dtype=torch.bfloat16, device="cuda")
        opt = AdamW([p], [c], state_bits=bits, max_norm=1.0)
        good, bad = torch.randn(1000, device="cuda"), torch.randn(1000, device="cuda")
        bad[999] = math.inf
        opt.step([good])
        keep = [t.clone() for t in (p, c, opt.m.view(torch.uint8), opt.v.view(torch.uint8), opt.steps)]
        assert opt.step([bad]).isinf()
        for a, b in zip((p, c, opt.m.view(torch.uint8), opt.v.view(torch.uint8), opt.steps), keep):
            assert torch.equal(a, b)
        opt.step([good])
        assert opt.steps.tolist() == [2, 0]


def test_blocks_that_are_not_finite_show_and_stay_within_their_block():
    p = torch.zeros(512, device="cuda")
    opt = AdamW([p], state_bits=8)
    g = torch.ones(512, device="cuda")
    g[200] = math.nan
    opt.step([g])
    bad = opt.m.float().isnan()
    assert bad[128:256].all() and not bad[:128].any() and not bad[256:].any()
    assert torch.equal(opt.v.float().isnan(), bad)
    assert p.isnan().nonzero().view(-1).tolist() == [200]


def test_small_roots_are_not_lost():
    """r's codes are at least 1 where v > 0: the next update stays bounded."""
    p = torch.zeros(128, device="cuda")
    opt = AdamW([p], lr=1.0, state_bits=8)
    g = torch.full((128,), 1e-9, device="cuda")
    g[0] = 1.0
    opt.step([g])
    assert (opt.v.view(torch.uint8) > 0).all()
    before = p.clone()
    opt.step([torch.zeros(128, device="cuda")])
    assert (p - before).abs().max() <= 2.0


def test_rounding_is_right_on_average():
    """Over many steps of no change (beta 1 - 2^-20, gradients that keep v and m
    where they are) the mean of the codes stays: each draw is off by at most one
    step of 1/8, so the mean over n of them by 1/8 * 5 / sqrt(n)."""
    n = 1 << 16
    gen = torch.Generator().manual_seed(5)
    p = torch.zeros(n, device="cuda")
    x = (1.0 + torch.rand(n, generator=gen))
    x.view(-1, 128)[:, 0] = 2.0                     # each block's largest value
    opt = AdamW([p], lr=0.0, betas=(0.0, 0.0), state_bits=8, seed=1)
    sums = [0.0, 0.0]
    for k in range(8):
        opt.step([x.cuda()])                        # m = g, r = |g|: rounded afresh in each step
        for j, (c, s) in enumerate(((opt.m, opt.m_scale), (opt.v, opt.v_scale))):
            got = (c.float().view(-1, 128) * s[:, None]).view(-1).cpu().double()
            assert ((got - x).abs() <= x / 8 + 1e-6).all()
            sums[j] += float((got - x).mean()) / 8
    for s in sums:
        assert abs(s) <= 0.25 / 8 * 2 * 5 / math.sqrt(8 * n) + 1e-6


def test_the_same_bits_every_time_and_after_a_restart():
    gen = torch.Generator().manual_seed(6)
    sizes = [5000, 77, 128]
    start = [torch.randn(n, generator=gen).cuda() for n in sizes]
    grads = [gradients(sizes, ("fp8", "bf16", "f32"), gen) for _ in range(4)]
    for bits in (8, 32):
        runs = []
        for split in (None, 2):
            params = [t.clone() for t in start]
            opt = AdamW(params, state_bits=bits, max_norm=0.5, seed=3)
            for k, g in enumerate(grads):
                if k == split:
                    saved = opt.state_dict()
                    opt = AdamW(params, state_bits=bits, max_norm=0.5, seed=3)
                    opt.load_state_dict(saved)
                opt.step(g)
            runs.append([t.clone() for t in params] + [opt.m.view(torch.uint8), opt.v.view(torch.uint8), opt.steps])
        assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_steps_count_themselves(bits):
    gen = torch.Generator().manual_seed(8)
    sizes = [3000, 129]
    start = [torch.randn(n, generator=gen).cuda() for n in sizes]
    grads = [torch.randn(n, generator=gen).cuda() for n in sizes]
    factor = torch.ones(1, device="cuda")
    eager, graphed = ([t.clone() for t in start] for _ in range(2))
    a, b = AdamW(eager, state_bits=bits, max_norm=1.0), AdamW(graphed, state_bits=bits, max_norm=1.0)
    for k in range(2):
        a.step(grads, lr_factor=factor)
    b.step(grads, lr_factor=factor)
    b.step(grads, lr_factor=factor)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = b.step(grads, lr_factor=factor)
    assert torch.equal(graphed[0], eager[0])        # capturing does nothing
    for k in range(3):
        for g in grads:
            g.mul_(0.9)
        factor.mul_(0.5)
        want = a.step(grads, lr_factor=factor)
        graph.replay()
        assert torch.equal(norm, want)
        assert all(torch.equal(x, y) for x, y in zip(eager, graphed)) and torch.equal(a.steps, b.steps)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step(grads, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b.step(grads)
    assert all(torch.equal(x, y) for x, y in zip(eager, graphed))
    assert api.taco_device_error() == 0


def test_elements_beyond_32_bits():
    """The hash and the offsets of a tensor with more than 2^32 values."""
    n, k = (1 << 32) + 4096 + 5, 5000
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = (1e-3 * torch.randn(k, generator=torch.Generator().manual_seed(9))).bfloat16()
    g[-k:] = tail.cuda()
    opt = AdamW([p], lr=1e-2, betas=BETAS, state_bits=8, max_norm=1e6, seed=11)
    norm = opt.step([g])
    want = float(tail.double().norm())
    assert abs(float(norm) - want) <= 40 * R.U * want
    (q, dq), (m, dm), _, _ = R.adamw(torch.zeros(k).double(), tail.double(), torch.zeros(k).double(),
                                     torch.zeros(k).double(), 1, float(np.float32(1e-2)), 0.0, *BETAS, EPS, 1.0, 2 * R.U)
    assert ((p[-k:].cpu().double() - q).abs() <= dq).all() and not p[:-k].any()
    skip = (-(n - k)) % 128                          # from the tail's first whole block on
    bits = R.bits_of(k - skip, 0, 0, 11, n - k + skip)
    lo, hi, sc, dsc = R.code_range(m[skip:], dm[skip:], bits & 0xFFFF, False)
    got = F.code_values(opt.m[n - k + skip:n].view(torch.uint8))
    assert ((lo <= got.abs()) & (got.abs() <= hi)).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_what_lies_around_the_tensors_is_left(bits):
    sizes = [1, 127, 515, 4097, 2048]
    place = [128 * i + sum(-(-n // 128) * 128 for n in sizes[:i]) for i in range(len(sizes))]
    total = place[-1] + sizes[-1] + 128
    p, c = torch.full((total,), 7.0, device="cuda"), torch.full((total,), 7.0, dtype=torch.bfloat16, device="cuda")
    part = lambda t: [t[a + 64:a + 64 + n] for a, n in zip(place, sizes)]
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    for t in part(inside):
        t.fill_(True)
    opt = AdamW(part(p), part(c), lr=0.1, weight_decay=0.1, state_bits=bits, max_norm=1.0)
    opt.step([torch.ones(n, device="cuda") for n in sizes])
    assert (p[~inside] == 7.0).all() and (c[~inside] == 7.0).all()
    assert (p[inside] != 7.0).all() and torch.equal(c[inside], p[inside].bfloat16())


def test_a_tensor_with_other_memory_is_refused():
    p, g = torch.ones(256, device="cuda"), torch.ones(256, device="cuda")
    opt = AdamW([p])
    opt.step([g])
    with pytest.raises(_lib.TacoError):
        opt.step([p])                               # its own gradient
    p.data = torch.ones(256, device="cuda")
    with pytest.raises(RuntimeError):
        opt.step([g])
    assert opt.steps.tolist() == [1, 0]
