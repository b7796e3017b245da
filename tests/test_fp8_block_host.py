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
