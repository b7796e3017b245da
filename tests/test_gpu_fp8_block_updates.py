"""Fp8Block over several steps on the GPU: a gate for one call, and weights
quantised again after an update, give the bits of a block made with them."""

import pytest
import torch

from fp8_communication_compression_gb300 import Fp8Block, api

pytestmark = pytest.mark.gpu


def test_gates_and_updated_weights():
    P, T, d, f = 2, 70, 256, 512
    g = torch.Generator().manual_seed(81)
    r = lambda *s: torch.randn(s, generator=g)
    w = [((r(f, d) / d ** 0.5).bfloat16().cuda(), (r(d, f) / f ** 0.5).bfloat16().cuda()) for _ in range(2)]
    y, h, dout, dh1 = (r(T, d).bfloat16().cuda() for _ in range(4))
    gates = [(0.5 + 0.1 * r(d)).cuda(), torch.sigmoid(r(T, 1)).cuda()]

    def step(block, gate=None):
        out, h1 = block.forward(y, h) if gate is None else block.forward(y, h, gate)
        return (out, h1, *block.backward(dout, dh1))

    want = step(Fp8Block(*w[1], T, P, gate=gates[1]))
    block = Fp8Block(*w[0], T, P, gate=gates[0])
    step(block)
    before = [m[0].clone() for m in block.main_up]
    block.load_weights(*w[1])
    assert all(torch.equal(m[0], b) for m, b in zip(block.main_up, before))
    got = step(block, gates[1])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not any(torch.equal(m[0], b) for m, b in zip(block.main_up, before))
    assert api.taco_device_error(clear=True) == 0
