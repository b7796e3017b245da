"""The FP8 block: everything the layer is made of, run together, against the
same block in float64 without any quantisation.

An E4M3 value is off by at most 2^-4 of itself, evenly spread inside its
step: 2^-4 / sqrt(3) rms at most, 3.6 %.  A product's terms carry two such
errors (5.1 % rms each, independent, so the sum's relative error is the same),
and a result passes through at most four quantised products or compressed
sums in a row: 0.051 * sqrt(4) + 0.036 = 0.14 of its norm bounds it."""

import pytest
import torch

import fp8_reference as R
from fp8_communication_compression_gb300 import api
from fp8_communication_compression_gb300.fp8_block import Fp8Block

pytestmark = pytest.mark.gpu

BOUND = 0.14


def rel(a, b):
    return ((a.cpu().double() - b).norm() / b.norm()).item()


def decode(codes, mult):
    m = mult.cpu().double().repeat_interleave(128).view(codes.shape)
    return R.code_values(codes) * m


@pytest.mark.parametrize("P,T,d,f", [(1, 64, 256, 512), (2, 200, 384, 1024)])
def test_block_against_float64(P, T, d, f):
    g = torch.Generator().manual_seed(P)
    r = lambda *s: torch.randn(s, generator=g)
    w_up, w_down = (r(f, d) / d ** 0.5).bfloat16().cuda(), (r(d, f) / f ** 0.5).bfloat16().cuda()
    y, h, dout, dh1 = (r(T, d).bfloat16().cuda() for _ in range(4))
    gate = (0.5 + 0.1 * r(d)).cuda()
    block = Fp8Block(w_up, w_down, T, P, gate=gate, residual_scale=0.9)
    out, h1 = block.forward(y, h)
    dy, dh, dgp, dgq, dgate = block.backward(dout, dh1)

    t = {k: v.cpu().double().requires_grad_() for k, v in
         dict(y=y, h=h, up=w_up, down=w_down, gp=block.gain_post, gq=block.gain_pre, gate=gate).items()}
    z = t["y"] / (t["y"].square().mean(1, keepdim=True) + 1e-6).sqrt() * t["gp"]
    rh = 0.9 * t["h"] + t["gate"] * z
    n = rh / (rh.square().mean(1, keepdim=True) + 1e-6).sqrt() * t["gq"]
    ref = torch.nn.functional.silu(n @ t["up"].t()) @ t["down"].t()
    loss = (ref * dout.cpu().double()).sum() + (rh * dh1.cpu().double()).sum()
    grads = torch.autograd.grad(loss, [t[k] for k in ("y", "h", "gp", "gq", "gate", "up", "down")])
    assert rel(out, ref.detach()) <= BOUND
    assert rel(h1, rh.detach()) <= 2.0 ** -8
    for got, want in zip((dy, dh, dgp, dgq, dgate), grads[:5]):
        assert rel(got, want) <= BOUND
    up = torch.cat([decode(*m) for m in block.main_up], 0)
    down = torch.cat([decode(*m) for m in block.main_down], 1)
    assert rel(up, grads[5]) <= BOUND and rel(down, grads[6]) <= BOUND

    # the same bits every time, and a second micro-batch adds to the first
    out2, _ = block.forward(y, h)
    again = block.backward(dout, dh1)
    assert torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip((dy, dh, dgp, dgq, dgate), again))
    up2 = torch.cat([decode(*m) for m in block.main_up], 0)
    assert rel(up2, 2 * grads[5]) <= BOUND
    assert api.taco_device_error(clear=True) == 0
