"""Fp8Block's order of calls without a GPU: the library's calls are replaced by
ones that note that they were made."""

import pytest
import torch

from fp8_communication_compression_gb300 import Fp8Block, api

T, D, F = 4, 128, 256


@pytest.fixture()
def block(monkeypatch):
    calls = []
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)

    def note(name, value):
        def call(*args, **kw):
            calls.append((name, args, kw))
            return value(*args, **kw)
        monkeypatch.setattr(api, name, call)

    note("fp8_quantize_weight", lambda w: (w, "scale", w.t(), "scale_t"))
    note("rmsnorm_gate_residual_fp8", lambda *a: (z(T, D), "codes", "scale"))
    note("rmsnorm_gate_residual", lambda *a: (z(T, D), z(T, D)))
    note("rmsnorm_gate_residual_backward", lambda *a: (z(T, D),) * 2 + (torch.zeros(D),) * 2 + (None,))
    note("fp8_gemm", lambda c, s, w, ws: z(T, F))
    note("fp8_linear", lambda x, w, s: z(T, D))
    note("fp8_linear_backward", lambda dy, x, ct, st, dw_dtype: (z(*x.shape), z(dy.shape[1], x.shape[1])))
    note("agoq_fp8_accumulate", lambda codes, scale, dw: None)

    class Sum:
        def __init__(self, *args, **kw):
            pass

        def run(self, x):
            return x.sum(0)

    monkeypatch.setattr(api, "TwoShotLocal", Sum)
    b = Fp8Block(z(F, D), z(D, F), T, gate=torch.ones(D))
    calls.clear()
    return b, calls


def named(calls, name):
    return [c for c in calls if c[0] == name]


def test_each_backward_pass_takes_its_own_forward_pass(block):
    b, calls = block
    x = torch.zeros((T, D), dtype=torch.bfloat16)
    with pytest.raises(RuntimeError):
        b.backward(x, x)
    b.forward(x, x)
    b.backward(x, x)
    assert len(named(calls, "agoq_fp8_accumulate")) == 2
    # the same micro-batch must not be added to the main gradients again
    with pytest.raises(RuntimeError):
        b.backward(x, x)
    assert len(named(calls, "agoq_fp8_accumulate")) == 2
    b.forward(x, x)
    b.backward(x, x)
    assert len(named(calls, "agoq_fp8_accumulate")) == 4


def test_a_call_may_bring_its_own_gate(block):
    b, calls = block
    x, gate = torch.zeros((T, D), dtype=torch.bfloat16), torch.full((T, 1), 0.5)
    for given, used in ((gate, gate), (None, b.gate)):
        calls.clear()
        b.forward(x, x, given)
        b.backward(x, x)
        norms = [c for c in calls if c[0].startswith("rmsnorm")]
        assert len(norms) == 3 and all(any(a is used for a in args) for _, args, _ in norms)


def test_updated_weights_are_quantised_in_place_of_the_old_ones(block):
    b, calls = block
    x = torch.zeros((T, D), dtype=torch.bfloat16)
    main = [m[0] for m in (*b.main_up, *b.main_down)]
    up, down = torch.ones((F, D), dtype=torch.bfloat16), torch.ones((D, F), dtype=torch.bfloat16)
    b.load_weights(up, down)
    assert torch.equal(b.up[0][0], up) and torch.equal(b.down[0][0], down)
    assert all(m[0] is old for m, old in zip((*b.main_up, *b.main_down), main))
    with pytest.raises(ValueError):
        b.load_weights(down, up)
    b.forward(x, x)
    b.load_weights(up, down)
    with pytest.raises(RuntimeError):
        b.backward(x, x)                  # that forward pass used the old ones
    b.forward(x, x)
    b.backward(x, x)
