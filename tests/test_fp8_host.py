"""The block-scaled FP8 calls and the norms around a block without a GPU:
argument checks (the pointers are never dereferenced), the binding's
refusals, and the tests' own float64 forms against independent facts."""

import ctypes
import itertools
import math

import pytest
import torch

import fp8_reference as R
from fp8_communication_compression_gb300 import _lib, api

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
A = 1 << 24  # fake, aligned "device addresses", far apart; never dereferenced


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_pitch(lib):
    for n in (0, 1, 15, 16, 17, 4096, 4097):
        assert lib.fp8_pitch(n) == api.fp8_pitch(n) == -(-n // 16) * 16


def test_scale_bytes_and_their_plain_order(lib):
    for rows, cols in ((1, 1), (128, 512), (129, 513), (300, 2560)):
        assert lib.fp8_scale_bytes(rows, cols) == -(-rows // 128) * -(-cols // 512) * 512
        assert math.prod(api._scale_shape(rows, cols)) == lib.fp8_scale_bytes(rows, cols)


@pytest.mark.parametrize("fn", ["fp8_quantize", "fp8_quantize_weight"])
def test_quantize_validation(lib, fn):
    f = lambda x=A, rows=64, cols=256, c=A * 2, s=A * 3, ct=A * 4, st=A * 5: getattr(lib, fn)(
        x, rows, cols, c, s, ct, st, None)
    assert f(rows=-1) == INVALID and f(cols=-1) == INVALID
    assert f(rows=0) == OK and f(cols=0) == OK
    assert f(rows=(1 << 30) + 1) == UNSUPPORTED and f(cols=(1 << 30) + 1) == UNSUPPORTED
    assert f(rows=1 << 30, cols=1 << 30) == UNSUPPORTED       # more tiles than the grid holds
    assert f(x=None) == INVALID
    assert f(c=None) == INVALID and f(st=None) == INVALID     # half a direction
    assert f(c=None, s=None, ct=None, st=None) == INVALID     # nothing to do
    assert f(x=A + 8) == MISALIGNED and f(c=A * 2 + 8) == MISALIGNED and f(ct=A * 4 + 4) == MISALIGNED
    assert (f(s=A * 3 + 8) == MISALIGNED) == (fn == "fp8_quantize")
    assert f(c=A) == INVALID                                  # codes over the input
    assert f(s=A * 2 + 64 * 256 - 16) == INVALID              # scales over the last codes
    assert f(ct=A * 2 + 16) == INVALID                        # the two code matrices overlap


def test_gemm_validation(lib):
    f = lambda **k: lib.fp8_gemm(k.get("a", A), k.get("sa", A * 2), k.get("b", A * 3), k.get("sb", A * 4),
                                 k.get("t", 0), k.get("M", 32), k.get("N", 64), k.get("K", 256), k.get("o", A * 5),
                                 k.get("bf", 1), None)
    assert f(M=-1) == INVALID and f(N=-1) == INVALID and f(K=-16) == INVALID
    assert f(K=100) == INVALID                                # rows of codes come in 16s
    assert f(M=0) == OK and f(N=0) == OK
    assert f(M=(1 << 30) + 1) == UNSUPPORTED
    for k in ("a", "sa", "b", "sb", "o"):
        assert f(**{k: None}) == INVALID
    for k in ("a", "sa", "b", "sb", "o"):
        assert f(**{k: A * 7 + 8}) == MISALIGNED
    for at in (A, A * 2, A * 3, A * 4):
        assert f(o=at) == INVALID                             # output over an input


def test_linear_validation(lib):
    v = ctypes.c_uint64(1)
    assert lib.fp8_linear_workspace_bytes(32, 64, 256, 0, None) == INVALID
    assert lib.fp8_linear_workspace_bytes(-1, 64, 256, 0, ctypes.byref(v)) == INVALID
    assert lib.fp8_linear_workspace_bytes(32, 64, (1 << 30) + 1, 0, ctypes.byref(v)) == UNSUPPORTED
    assert lib.fp8_linear_workspace_bytes(32, 64, 256, 0, ctypes.byref(v)) == OK
    need = v.value
    assert need >= 32 * 256 + 2 * 32
    f = lambda **k: lib.fp8_linear(k.get("x", A), k.get("c", A * 2), k.get("s", A * 3), k.get("M", 32),
                                   k.get("N", 64), k.get("K", 256), k.get("y", A * 4), 1, k.get("ws", A * 5),
                                   k.get("n", need), None)
    assert f(M=0) == OK and f(N=0) == OK
    assert f(M=-1) == INVALID
    for k in ("x", "c", "s", "y", "ws"):
        assert f(**{k: None}) == INVALID
    assert f(n=need - 1) == INVALID                           # workspace too small
    assert f(x=A + 2) == MISALIGNED and f(ws=A * 5 + 128) == MISALIGNED and f(y=A * 4 + 8) == MISALIGNED
    assert f(ws=A) == INVALID and f(y=A * 2) == INVALID and f(y=A * 5) == INVALID

    assert lib.fp8_linear_workspace_bytes(32, 64, 256, 1, ctypes.byref(v)) == OK
    nb = v.value
    b = lambda **k: lib.fp8_linear_backward(k.get("dy", A), k.get("x", A * 2), k.get("c", A * 3), k.get("s", A * 4),
                                            k.get("M", 32), k.get("N", 64), k.get("K", 256), k.get("dx", A * 5),
                                            k.get("dw", A * 6), 0, k.get("ws", A * 7), k.get("n", nb), None)
    assert b(dx=None, dw=None) == INVALID
    assert b(K=0) == OK
    assert b(M=0, dw=None) == OK                              # no rows of dx
    for k in ("dy", "x", "c", "s", "ws"):
        assert b(**{k: None}) == INVALID
    assert b(n=nb - 1) == INVALID
    assert b(dy=A + 2) == MISALIGNED and b(dw=A * 6 + 4) == MISALIGNED and b(ws=A * 7 + 16) == MISALIGNED
    assert b(dx=A * 6) == INVALID and b(dw=A * 2) == INVALID and b(dx=A * 7) == INVALID


def test_norm_validation(lib):
    f = lambda **k: lib.rmsnorm_gate_residual(k.get("y", A), k.get("h", A * 2), k.get("gp", A * 3), k.get("gq", A * 4),
                                              k.get("g", None), k.get("mode", 0), k.get("s", 1.0),
                                              k.get("eps", 1e-6), k.get("T", 8), k.get("d", 256),
                                              k.get("o", A * 6), k.get("n", A * 7), k.get("ns", None), None)
    assert f(T=-1) == INVALID and f(d=0) == INVALID and f(d=-8) == INVALID
    assert f(d=16385) == UNSUPPORTED
    assert f(T=0) == OK
    assert f(mode=4) == INVALID and f(mode=-1) == INVALID
    assert f(mode=1) == INVALID and f(mode=0, g=A * 5) == INVALID  # gate and mode disagree
    for e in (0.0, -1.0, math.nan, math.inf):
        assert f(eps=e) == INVALID
    assert f(s=math.nan) == INVALID and f(s=math.inf) == INVALID
    for k in ("y", "h", "gp", "gq", "o", "n"):
        assert f(**{k: None}) == INVALID
        assert f(**{k: A * 9 + 8}) == MISALIGNED
    assert f(mode=3, g=A * 5 + 8) == MISALIGNED and f(mode=2, g=A * 5 + 2) == MISALIGNED
    assert f(o=A) == INVALID and f(n=A * 6 + 16) == INVALID and f(mode=1, g=A * 6) == INVALID
    assert f(ns=A * 7 + 8 * 256 - 16) == INVALID               # scales over the codes
    assert f(ns=A * 8 + 8) == MISALIGNED

    v = ctypes.c_uint64(0)
    assert lib.rmsnorm_gate_residual_workspace_bytes(8, 256, 0, None) == INVALID
    assert lib.rmsnorm_gate_residual_workspace_bytes(8, 0, 0, ctypes.byref(v)) == INVALID
    assert lib.rmsnorm_gate_residual_workspace_bytes(0, 256, 0, ctypes.byref(v)) == OK and v.value == 0
    b = lambda **k: lib.rmsnorm_gate_residual_backward(
        k.get("dn", A), k.get("dho", A * 2), k.get("y", A * 3), k.get("h", A * 4), k.get("gp", A * 5),
        k.get("gq", A * 6), k.get("g", None), k.get("mode", 0), k.get("s", 1.0), k.get("eps", 1e-6), k.get("T", 8),
        k.get("d", 256), k.get("dy", A * 8), k.get("dh", A * 9), k.get("dgp", A * 10), k.get("dgq", A * 11),
        k.get("dg", None), k.get("ws", A * 13), k.get("n", 1 << 22), None)
    assert b(T=-1) == INVALID and b(d=16385) == UNSUPPORTED and b(eps=0.0) == INVALID
    for k in ("dn", "dho", "y", "h", "gp", "gq", "dy", "dh", "dgp", "dgq", "ws"):
        assert b(**{k: None}) == INVALID
    assert b(mode=1, g=A * 7) == INVALID                       # no room for the gate's gradient
    assert b(dg=A * 12) == INVALID                             # a gradient of no gate
    assert b(dn=A + 8) == MISALIGNED and b(ws=A * 13 + 16) == MISALIGNED


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.fp8_quantize(x)
    with pytest.raises(ValueError, match="CUDA"):
        api.rmsnorm_gate_residual(x, x, torch.ones(64), torch.ones(64))
    with pytest.raises(TypeError):
        api.fp8_linear([1.0], x, x)


def test_block_exponent_is_the_smallest_that_fits():
    a = torch.tensor([0.0, 448.0, 448.0001, 449.0, 1.0, 2.0 ** -133, 3.3e38, 0.875, 0.8750001], dtype=torch.float64)
    E = R.block_exponent(a)
    for v, e in zip(a.tolist(), E.tolist()):
        if v == 0:
            assert e == 0
        else:
            assert v <= 448 * 2.0 ** e and (e == -127 or v > 448 * 2.0 ** (e - 1))


def test_e4m3_round_is_the_nearest_code():
    vals = R.code_values(torch.arange(256))
    fin = vals[torch.isfinite(vals)].unique()
    v = torch.linspace(-448, 448, 20011, dtype=torch.float64)
    v = torch.cat([v, v * 2.0 ** -9, fin, (fin[1:] + fin[:-1]) / 2])
    got = R.e4m3_round(v)
    assert torch.isin(got, fin).all()
    best = (v[:, None] - fin[None]).abs().amin(1)
    assert torch.equal((got - v).abs(), best)


@pytest.mark.parametrize("mode", ["none", "channel", "token", "full"])
def test_norm_gradients_against_differences(mode):
    g = torch.Generator().manual_seed(3)
    T, d, s, eps = 3, 7, 0.7, 1e-3
    r = lambda *sh: torch.randn(sh, generator=g, dtype=torch.float64)
    y, h, gp, gq, dn, dh2 = r(T, d), r(T, d), r(d), r(d), r(T, d), r(T, d)
    gate = {"none": None, "channel": r(d), "token": r(T, 1), "full": r(T, d)}[mode]

    def loss(y, h, gp, gq, gate):
        h2, n = R.norm_forward(y, h, gp, gq, gate, s, eps)
        return (h2 * dh2).sum() + (n * dn).sum()

    h2, _ = R.norm_forward(y, h, gp, gq, gate, s, eps)
    dy, dh, dgp, dgq, dgate = R.norm_backward(dn, dh2, y, h2, gp, gq, gate.float() if mode == "token" else gate,
                                              s, eps)
    args = [y, h, gp, gq] + ([] if gate is None else [gate])
    grads = [dy, dh, dgp, dgq] + ([] if gate is None else [dgate])
    tol = 1e-5 if mode == "token" else 1e-7  # (the token gate goes in as fp32)
    step = 1e-5
    for k, (a, ga) in enumerate(zip(args, grads)):
        for idx in itertools.islice(itertools.product(*[range(n) for n in a.shape]), 12):
            v = []
            for sg in (1, -1):
                b = a.clone()
                b[idx] += sg * step
                full = args[:k] + [b] + args[k + 1:]
                v.append(loss(*full, *([None] if gate is None else [])))
            assert abs((v[0] - v[1]) / (2 * step) - ga[idx]) <= tol * (1 + abs(ga[idx])), (mode, k, idx)


def test_block_refuses_shapes_that_do_not_divide():
    from fp8_communication_compression_gb300 import Fp8Block

    w = lambda r, c: torch.zeros((r, c), dtype=torch.bfloat16)
    for up, down, tokens, P in ((w(256, 100), w(100, 256), 8, 1), (w(256, 128), w(256, 128), 8, 1),
                                (w(256, 128), w(128, 256), 8, 3), (w(256, 128), w(128, 256), 0, 2)):
        with pytest.raises(ValueError):
            Fp8Block(up, down, tokens, P)
