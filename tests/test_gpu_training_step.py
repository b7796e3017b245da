"""One training step with all of it: Fp8Block, Fp8Head with a loss, FP8 main
gradients, their norm, AdamW, and the new weights quantised again."""

import math

import numpy as np
import pytest
import torch

import training_reference as R
from fp8_communication_compression_gb300 import AdamW, Fp8Block, Fp8Head, api
from test_gpu_adamw import state_values, values

pytestmark = pytest.mark.gpu

T, D, F, P, VOCAB = 192, 256, 512, 2, 500


def model(seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).cuda()
    up = [r(F // P, D) / math.sqrt(D) for _ in range(P)]
    down = [r(D, F // P) / math.sqrt(F) for _ in range(P)]
    head = r(512, D) / math.sqrt(D)
    head[VOCAB:] = 0.0
    gain = torch.ones(D, device="cuda")
    return [*up, *down, head, gain], r


def weights(copies):
    return torch.cat(copies[:P]), torch.cat(copies[P:2 * P], 1), copies[2 * P]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_steps(bits, loss):
    params, r = model()
    copies = [p.bfloat16() for p in params[:-1]] + [None]
    up, down, w = weights(copies)
    block, head = Fp8Block(up, down, T, P), Fp8Head(w[:VOCAB].contiguous())
    block.gain_pre = params[-1]
    opt = AdamW(params, copies, lr=1e-3, weight_decay=[0.1] * (2 * P + 1) + [0.0], state_bits=bits, max_norm=0.5, seed=5)
    y, h = r(T, D).bfloat16(), r(T, D).bfloat16()
    a = torch.randint(0, VOCAB, (T,), generator=torch.Generator().manual_seed(2)).cuda()
    a[:10] = -1
    offsets = torch.tensor([0, 50, 90, 150, 180]).cuda()
    for k in range(2):
        out, h1 = block.forward(y, h)
        logits = head.logits(out)
        assert logits.shape == (T, 512) and not logits[:, VOCAB:].any()
        if loss == "policy":
            old = head.token_logprob(out, a, 0.9) - 0.05
            adv, wt = r(T), torch.full((T,), 1.0 / T, device="cuda")
            want = R.policy(logits, a, old, adv, wt, old, 0.2, 0.2, 0.1, VOCAB, 0.9)
            got, dx = head.policy_loss(out, a, old, adv, wt, ref_logp=old, kl=0.1, temperature=0.9)
        else:
            ref = head.token_logprob(out, a) + 0.1 * r(T)
            want = R.preference(logits, a, offsets, ref, 0.5, 0.1, False, VOCAB, 1.0)
            got, dx = head.preference_loss(out, a, offsets, ref, beta=0.5, label_smoothing=0.1)
        for name, (value, tol) in want.items():
            assert ((getattr(got, name).cpu().double().reshape(value.shape) - value).abs() <= tol).all(), name
        dy, dh, dg_post, dg_pre, _ = block.backward(dx, torch.zeros_like(h1))
        grads = [*block.gradients(), head.main, dg_pre]
        assert all(values(g).isfinite().all() and values(g).any() for g in grads)
        before = [(p.cpu().double().view(-1), *state_values(opt, i)) for i, p in enumerate(params)]
        norm = float(opt.step(grads))
        want_norm = math.sqrt(sum(float(values(g).square().sum()) for g in grads))
        assert abs(norm - want_norm) <= 40 * R.U * want_norm
        coef = min(1.0, 0.5 / (want_norm + 1e-6))
        for i, (p, g) in enumerate(zip(params, grads)):
            wd = float(np.float32(0.1)) if i < 2 * P + 1 else 0.0
            (q, dq), *_ = R.adamw(before[i][0], values(g), before[i][1], before[i][2], k + 1, float(np.float32(1e-3)), wd,
                                  0.9, 0.95, 1e-8, coef, 46 * R.U)
            assert ((p.cpu().double().view(-1) - q).abs() <= dq).all(), i
            assert copies[i] is None or torch.equal(copies[i], p.bfloat16())
        assert not params[2 * P][VOCAB:].any()          # the padding stays zero
        up, down, w = weights(copies)
        block.load_weights(up, down)
        head.load_weights(w)
        block.zero_gradients()
        head.zero_gradients()
        assert not any(values(g).any() for g in grads[:-1])
        assert torch.equal(head.w[0], api.fp8_quantize_weight(w)[0])
    assert opt.steps.tolist() == [2, 0] and api.taco_device_error() == 0


def test_a_captured_step():
    """The loss, its gradient, the layer's backward pass and the update replayed
    from one graph give what the calls give."""
    results = []
    for captured in (False, True):
        params, r = model(3)
        head_w = [params[2 * P]]
        copy = [head_w[0].bfloat16()]
        head = Fp8Head(copy[0][:VOCAB].contiguous())
        opt = AdamW(head_w, copy, lr=1e-2, state_bits=8, max_norm=1.0)
        x = r(T, D).bfloat16()
        a = torch.randint(0, VOCAB, (T,), generator=torch.Generator().manual_seed(4)).cuda()
        adv, wt, old = r(T), torch.full((T,), 1.0 / T, device="cuda"), torch.full((T,), -6.2, device="cuda")

        def step():
            got, dx = head.policy_loss(x, a, old, adv, wt)
            opt.step([head.main])
            head.zero_gradients()
            return got.loss, dx

        if captured:
            keep = [t.clone() for t in (head.main[0], head.main[1], head_w[0], copy[0])]
            for _ in range(2):
                step()
            torch.cuda.synchronize()
            for t, k in zip((head.main[0], head.main[1], head_w[0], copy[0]), keep):
                t.copy_(k)
            opt.load_state_dict(AdamW([torch.empty_like(head_w[0])], state_bits=8).state_dict())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                loss, dx = step()
            for _ in range(3):
                graph.replay()
        else:
            for _ in range(3):
                loss, dx = step()
        torch.cuda.synchronize()
        results.append([t.clone() for t in (loss, dx, head_w[0], copy[0], opt.m.view(torch.uint8), opt.steps)])
    assert all(torch.equal(p, q) for p, q in zip(*results))
