"""The losses over the vocabulary, grad_norm and AdamW without a GPU: argument
checks (the pointers are never dereferenced), the binding's refusals, Fp8Head's
order of calls, the rounding hash, and the tests' own float64 forms."""

import ctypes
import math

import numpy as np
import pytest
import torch

import training_reference as R
from fp8_communication_compression_gb300 import AdamW, Fp8Head, _lib, api

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
A = 1 << 24  # fake, aligned "device addresses", far apart; never dereferenced


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_logprob_validation(lib):
    f = lambda **k: lib.token_logprob(k.get("x", A), 1, k.get("a", A * 2), k.get("T", 4), k.get("V", 100),
                                      k.get("N", 128), k.get("tau", 1.0), k.get("p", A * 3), k.get("l", A * 4), None)
    assert f(T=-1) == INVALID and f(V=0) == INVALID and f(V=129) == INVALID
    assert f(T=0) == OK
    for tau in (0.0, -1.0, math.inf, math.nan, 1e-45):
        assert f(tau=tau) == INVALID
    assert f(T=1 << 31) == UNSUPPORTED and f(N=(1 << 31) - 63) == UNSUPPORTED
    for k in ("x", "a", "p", "l"):
        assert f(**{k: None}) == INVALID
        assert f(**{k: A * 7 + 2}) == MISALIGNED
    assert f(x=A + 8) == MISALIGNED
    assert f(p=A + 64) == INVALID and f(l=A * 3) == INVALID and f(l=A * 2) == INVALID
    g = lambda **k: lib.token_logprob_backward(k.get("d", A * 5), k.get("x", A), 0, k.get("a", A * 2), k.get("l", A * 4),
                                               k.get("T", 4), k.get("V", 100), 128, 1.0, k.get("o", A * 6), None)
    assert g(T=0) == OK and g(V=0) == INVALID
    for k in ("x", "a", "d", "l", "o"):
        assert g(**{k: None}) == INVALID
        assert g(**{k: A * 7 + 2}) == MISALIGNED
    assert g(o=A + 16) == INVALID and g(o=A * 2) == INVALID and g(o=A * 5) == INVALID


def test_policy_validation(lib):
    f = lambda **k: lib.policy_loss(k.get("x", A), 1, k.get("a", A * 2), k.get("old", A * 3), k.get("adv", A * 4),
                                    k.get("w", A * 5), k.get("ref", A * 6), k.get("T", 4), 100, 128, k.get("tau", 1.0),
                                    k.get("lo", 0.2), k.get("hi", 0.2), k.get("kl", 0.1), k.get("gs", 1.0),
                                    k.get("loss", A * 7), k.get("tl", A * 8), k.get("lp", A * 9), k.get("d", A * 10), None)
    for bad in (dict(lo=-0.1), dict(lo=1.1), dict(hi=-0.1), dict(hi=math.inf), dict(kl=math.nan), dict(gs=math.inf),
                dict(lo=math.nan), dict(tau=0.0), dict(ref=None), dict(T=-1)):
        assert f(**bad) == INVALID
    for k in ("x", "a", "old", "adv", "w", "loss", "tl", "lp"):
        assert f(**{k: None}) == INVALID
        assert f(**{k: A * 12 + 2}) == MISALIGNED
    assert f(d=A * 12 + 8) == MISALIGNED
    assert f(d=A + 16) == INVALID                 # part of the logits
    assert f(tl=A) == INVALID and f(lp=A * 8) == INVALID and f(loss=A * 5 + 4) == INVALID


def test_preference_validation(lib):
    v = ctypes.c_uint64(1)
    assert lib.preference_loss_workspace_bytes(4, 0, ctypes.byref(v)) == INVALID
    assert lib.preference_loss_workspace_bytes(-1, 1, ctypes.byref(v)) == INVALID
    assert lib.preference_loss_workspace_bytes(4, 1, None) == INVALID
    assert lib.preference_loss_workspace_bytes(1 << 31, 1, ctypes.byref(v)) == UNSUPPORTED
    assert lib.preference_loss_workspace_bytes(4, 2, ctypes.byref(v)) == OK and v.value == 4 * (12 + 2)
    f = lambda **k: lib.preference_loss(k.get("x", A), 1, k.get("a", A * 2), k.get("off", A * 3), k.get("ref", A * 4),
                                        k.get("T", 4), 100, 128, k.get("pairs", 2), 1.0, k.get("beta", 0.1),
                                        k.get("ls", 0.0), 0, k.get("gs", 1.0), k.get("loss", A * 5), k.get("m", A * 6),
                                        k.get("r", A * 7), k.get("lp", A * 8), k.get("d", A * 9), k.get("ws", A * 10),
                                        k.get("n", 56), None)
    for bad in (dict(pairs=0), dict(ls=-0.1), dict(ls=1.1), dict(ls=math.nan), dict(beta=math.inf), dict(gs=math.nan),
                dict(n=55), dict(T=-1)):
        assert f(**bad) == INVALID
    for k in ("x", "a", "off", "loss", "m", "r", "lp", "ws"):
        assert f(**{k: None}) == INVALID
        assert f(**{k: A * 12 + 2}) == MISALIGNED
    assert f(d=A + 16) == INVALID and f(ws=A) == INVALID and f(lp=A * 10) == INVALID and f(r=A * 3) == INVALID


def norm_call(lib, n=100, kind=0, grad=A, scale=None, norm=A * 2, ws=A * 3, nbytes=1 << 20, gs=1.0, count=1):
    t = (_lib.GradTensor * 1)(_lib.GradTensor(grad, scale, n, kind))
    return lib.grad_norm(t, count, gs, norm, ws, nbytes, None)


def test_grad_norm_validation(lib):
    v = ctypes.c_uint64(0)
    assert lib.grad_norm_workspace_bytes(1, None) == INVALID and lib.grad_norm_workspace_bytes(-1, ctypes.byref(v)) == INVALID
    assert lib.grad_norm_workspace_bytes(3, ctypes.byref(v)) == OK and v.value > 0
    f = lambda **k: norm_call(lib, **k)
    assert f(n=-1) == INVALID and f(kind=3) == INVALID and f(kind=2) == INVALID and f(scale=A * 4) == INVALID
    assert f(grad=None) == INVALID and f(norm=None) == INVALID and f(ws=None) == INVALID and f(nbytes=8) == INVALID
    assert f(gs=math.inf) == INVALID and f(count=-1) == INVALID
    assert f(n=(1 << 38) + 1) == UNSUPPORTED
    assert f(grad=A + 8) == MISALIGNED and f(norm=A * 2 + 2) == MISALIGNED and f(ws=A * 3 + 128) == MISALIGNED
    assert f(kind=2, scale=A * 4 + 2) == MISALIGNED
    assert f(norm=A + 16) == INVALID and f(ws=A) == INVALID and f(kind=2, scale=A * 2) == INVALID


def adamw_call(lib, count=1, bits=8, b1=0.9, b2=0.95, eps=1e-8, gs=1.0, norm=None, max_norm=0.0, factor=None,
               state=A * 10, ws=None, nbytes=0, **k):
    t = _lib.AdamWTensor(A, A * 2, A * 3, None, A * 4, A * 5, A * 6, A * 7, 100, 1e-3, 0.1, 0)
    for name, v in k.items():
        setattr(t, name, v)
    t = (_lib.AdamWTensor * 1)(t)
    return lib.adamw_step(t, count, bits, b1, b2, eps, gs, max_norm, norm, factor, 0, state, ws, nbytes, None)


def test_adamw_validation(lib):
    f = lambda **k: adamw_call(lib, **k)
    for bad in (dict(b1=1.0), dict(b2=-0.1), dict(b1=math.nan), dict(eps=0.0), dict(eps=1e-45), dict(eps=math.inf),
                dict(gs=math.nan), dict(max_norm=1.0), dict(max_norm=-1.0), dict(max_norm=math.inf, norm=A * 11),
                dict(count=-1), dict(n=-1), dict(lr=math.nan), dict(weight_decay=math.inf), dict(grad_type=5),
                dict(grad_type=2), dict(grad_scale=A * 8), dict(norm=A * 11), dict(state=None)):
        assert f(**bad) == INVALID, bad
    assert f(count=0) == OK
    assert f(bits=16) == UNSUPPORTED and f(n=(1 << 38) + 1) == UNSUPPORTED
    for name in ("param", "grad", "m", "v", "m_scale", "v_scale"):
        assert f(**{name: None}) == INVALID, name
    for name in ("param", "copy_bf16", "grad", "m", "v"):
        assert f(**{name: A * 12 + 8}) == MISALIGNED, name
    assert f(m_scale=A * 12 + 2) == MISALIGNED and f(state=A * 10 + 4) == MISALIGNED and f(factor=A + 2) == MISALIGNED
    for name, at in (("copy_bf16", A), ("m", A + 16), ("v", A * 4), ("m_scale", A * 7), ("grad", A), ("m", A * 3),
                     ("m", A * 10), ("param", A * 10)):
        assert f(**{name: at}) == INVALID, (name, at)
    assert f(factor=A) == INVALID
    big = dict(norm=A * 11, max_norm=1.0, ws=A * 13, nbytes=1 << 20)
    for name, at in (("norm", A), ("norm", A * 3), ("ws", A * 3), ("ws", A * 5), ("norm", A * 10), ("nbytes", 8)):
        assert f(**(big | {name: at})) == INVALID, (name, at)


class Fake(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


def t(shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Fake)


def test_the_binding_refuses_wrong_tensors():
    x, a, f = t((4, 32), torch.bfloat16), t(4, torch.int64), t(4)
    with pytest.raises(ValueError):
        api.token_logprob(torch.zeros(4, 32), a)                   # not on the GPU
    with pytest.raises(TypeError):
        api.token_logprob(x, t(4, torch.int32))
    with pytest.raises(TypeError):
        api.token_logprob(t((4, 32), torch.float16), a)
    with pytest.raises(ValueError):
        api.token_logprob(x, t(5, torch.int64))
    with pytest.raises(ValueError):
        api.token_logprob(x[:, ::2], a)
    for vocab in (0, 33):
        with pytest.raises(ValueError):
            api.token_logprob(x, a, vocab)
    with pytest.raises(ValueError):
        api.token_logprob(t(32), a)
    with pytest.raises(ValueError):
        api.policy_loss(x, a, f, f, f, kl=0.1)                      # no reference
    with pytest.raises(ValueError):
        api.policy_loss(x, a, f, f, f, need_grad=False, dlogits=x)
    with pytest.raises(TypeError):
        api.policy_loss(x, a, f, f, f, dlogits=t((4, 32)))
    with pytest.raises(ValueError):
        api.policy_loss(x, a, f, f, f, dlogits=t((8, 16), torch.bfloat16))
    for n in (1, 2, 4):
        with pytest.raises(ValueError):
            api.preference_loss(x, a, t(n, torch.int64))
    with pytest.raises(ValueError):
        api.token_logprob_backward(t(3), x, a, f)
    with pytest.raises(ValueError):
        api.grad_norm([])
    with pytest.raises(TypeError):
        api.grad_norm([t(4, torch.float16)])
    with pytest.raises(TypeError):
        api.grad_norm([t(4, torch.uint8)])                          # codes without a scale
    with pytest.raises(ValueError):
        api.grad_norm([(t(129, torch.uint8), t(1))])
    with pytest.raises(ValueError):
        api.grad_norm([t((4, 4)), t((4, 4))[:, :2]])


def test_adamw_refuses_wrong_arguments():
    p = lambda n=4: t(n)
    for args in (dict(params=[]), dict(copies=[]), dict(copies=[t(4)]), dict(lr=[1.0, 2.0]), dict(state_bits=16),
                 dict(betas=(1.0, 0.9)), dict(eps=0.0), dict(max_norm=0.0), dict(max_norm=-1.0),
                 dict(params=[t(4, torch.bfloat16)]), dict(copies=[t(5, torch.bfloat16)])):
        with pytest.raises((ValueError, TypeError)):
            AdamW(**({"params": [p()]} | args))
    q = p(8)
    with pytest.raises(ValueError):
        AdamW([q[:6], q[4:]])                                       # the same memory twice


def test_the_hash_is_uniform_and_independent():
    n = 1 << 18
    before = None
    for step in (0, 1, 1000):
        h = R.bits_of(n, 3, step, (5 << 32) + 77)
        halves = [(h & np.uint64(0xFFFF)).astype(np.float64) / 65536, (h >> np.uint64(16)).astype(np.float64) / 65536]
        for u in halves:
            assert abs(u.mean() - 0.5) <= 5 * math.sqrt(1 / 12 / n)
            counts = np.histogram(u, 64, (0, 1))[0]
            assert ((counts - n / 64) ** 2 / (n / 64)).sum() <= 63 + 6 * math.sqrt(2 * 63)
            for lag in (1, 2, 4, 32, 128):
                assert abs(np.corrcoef(u[:-lag], u[lag:])[0, 1]) <= 5 / math.sqrt(n)
        assert abs(np.corrcoef(*halves)[0, 1]) <= 5 / math.sqrt(n)
        if before is not None:
            assert abs(np.corrcoef(halves[0], before)[0, 1]) <= 5 / math.sqrt(n)
        before = halves[0]
    assert not np.array_equal(R.bits_of(8, 0, 0, 0), R.bits_of(8, 1, 0, 0))
    assert not np.array_equal(R.bits_of(8, 0, 0, 0), R.bits_of(8, 0, 0, 1 << 32))
    assert not np.array_equal(R.bits_of(8, 0, 0, 0), R.bits_of(8, 0, 0, 0, 1 << 32))


def test_reference_gradients_against_differences():
    """The float64 forms themselves: central differences, h^2 times a third
    derivative of order one, over step 1e-5: 1e-8."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn((5, 9), generator=g, dtype=torch.float64)
    a = torch.tensor([1, 8, -1, 3, 0])
    old, ref = (-2.0 + 0.3 * torch.randn(5, generator=g, dtype=torch.float64) for _ in range(2))
    adv, w = torch.randn(5, generator=g, dtype=torch.float64), torch.rand(5, generator=g, dtype=torch.float64)
    off = torch.tensor([0, 2, 4])
    forms = {"policy": lambda z: R.policy(z, a, old, adv, w, ref, 0.2, 0.3, 0.1, 8, 0.7),
             "preference": lambda z: R.preference(z, a, off, ref, 0.5, 0.1, True, 8, 0.7)}
    a[1] = 7
    for f in forms.values():
        d = f(x)["dlogits"][0]
        for t in range(5):
            for j in range(9):
                up, down = x.clone(), x.clone()
                up[t, j] += 1e-5
                down[t, j] -= 1e-5
                assert abs(float((f(up)["loss"][0] - f(down)["loss"][0]) / 2e-5 - d[t, j])) <= 1e-7


def test_head_gives_the_gradient_the_logits_place(monkeypatch):
    calls = []
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    monkeypatch.setattr(api, "fp8_quantize_weight", lambda w: (w, "s", w.t(), "st"))
    monkeypatch.setattr(api, "fp8_linear", lambda x, c, s: bf(x.shape[0], c.shape[0]))
    monkeypatch.setattr(api, "fp8_linear_backward", lambda dy, x, ct, st, dw_dtype: (calls.append(dy), (bf(*x.shape), bf(dy.shape[1], x.shape[1])))[1])
    monkeypatch.setattr(api, "agoq_fp8_accumulate", lambda codes, scale, dw: calls.append((codes, dw.shape)))
    seen = {}
    monkeypatch.setattr(api, "policy_loss", lambda logits, *a, **k: seen.update(k, logits=logits) or "loss")
    head = Fp8Head(bf(200, 128))
    assert head.rows == 256 and head.w[0].shape == (256, 128) and head.main[0].shape == (256, 128)
    got, dx = head.policy_loss(bf(5, 128), "a", "o", "adv", "w", kl=0.5, ref_logp="r")
    assert got == "loss" and dx.shape == (5, 128)
    assert seen["dlogits"] is seen["logits"] and seen["vocab"] == 200 and seen["kl"] == 0.5
    assert calls[0] is seen["logits"] and calls[1][0] is head.main[0] and calls[1][1] == (256, 128)
    head.load_weights(bf(256, 128))
    for wrong in (bf(128, 128), bf(200, 256)):
        with pytest.raises(ValueError):
            head.load_weights(wrong)
    with pytest.raises(ValueError):
        Fp8Head(bf(200, 100))
