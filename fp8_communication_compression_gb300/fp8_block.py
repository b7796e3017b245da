"""One MLP block trained in FP8, in P tensor-parallel slices on one GPU: the
norms around the block, its two linear layers, the compressed two-shot sum of
the slices' partial outputs, and the FP8 main gradients, run together.

    h1 = residual_scale * h + gate * rmsnorm(y) * gain_post     y: the block before
    n  = rmsnorm(h1) * gain_pre                                 written as FP8 codes
    u_p = n W_up_p^T;  a_p = silu(u_p);  s_p = a_p W_down_p^T   slice p of P
    out = sum_p s_p                                             TwoShotLocal: each
                                                                partial sum compressed

``out`` and ``h1`` go into the next block's norms.  The backward pass keeps
y, h1 and the u_p; n and the a_p are recomputed (AGoQ 2.A stores inputs and
recomputes).  Weight gradients go straight into FP8 main gradients
(agoq_fp8_accumulate), one micro-batch after the other.

It shows how the calls fit together.  What lies between them is plain torch
(SiLU and its gradient, the stacking of the partial sums), and the bf16 weight
gradient passes through memory on its way into the main gradients."""

from __future__ import annotations

import torch

from . import api


class Fp8Block:
    """``w_up`` bf16 [f, d] and ``w_down`` bf16 [d, f], f split into P equal
    slices; ``gate`` as rmsnorm_gate_residual's.  A gate that changes with the
    tokens is given to forward() instead."""

    def __init__(self, w_up: torch.Tensor, w_down: torch.Tensor, tokens: int, P: int = 1,
                 gate: torch.Tensor | None = None, residual_scale: float = 1.0, eps: float = 1e-6):
        f, d = w_up.shape
        if tuple(w_down.shape) != (d, f) or f % (128 * P) or d % 128:
            raise ValueError("w_up must be [f, d] and w_down [d, f], d a multiple of 128 and f of 128 P")
        if tokens < 1:
            raise ValueError("tokens must be positive")
        dev = w_up.device
        self.P, self.tokens, self.d, self.f = P, tokens, d, f
        self.gate, self.residual_scale, self.eps = gate, residual_scale, eps
        self.gain_post = torch.ones(d, device=dev)
        self.gain_pre = torch.ones(d, device=dev)
        fp = f // P
        self.load_weights(w_up, w_down)
        self.sum = api.TwoShotLocal(P, tokens, d, out_dtype=torch.bfloat16, device=dev)
        # FP8 main gradients of the slices' weights: codes and multipliers
        self.main_up = [self._main(fp, d, dev) for _ in range(P)]
        self.main_down = [self._main(d, fp, dev) for _ in range(P)]

    def load_weights(self, w_up: torch.Tensor, w_down: torch.Tensor) -> None:
        """Quantises each slice's weights: at the start, and after an update.
        The main gradients stay as they are; a forward pass with the old
        weights can no longer be followed by its backward pass."""
        if tuple(w_up.shape) != (self.f, self.d) or tuple(w_down.shape) != (self.d, self.f):
            raise ValueError(f"w_up must be [{self.f}, {self.d}] and w_down [{self.d}, {self.f}]")
        self._saved = None  # what the backward pass needs of the forward one
        fp = self.f // self.P
        self.up = [api.fp8_quantize_weight(w_up[p * fp:(p + 1) * fp]) for p in range(self.P)]
        self.down = [api.fp8_quantize_weight(w_down[:, p * fp:(p + 1) * fp].contiguous()) for p in range(self.P)]

    @staticmethod
    def _main(rows: int, cols: int, dev: torch.device):
        return (torch.zeros((rows, cols), dtype=torch.uint8, device=dev),
                torch.ones(rows * cols // 128, dtype=torch.float32, device=dev))

    def _reduce(self, parts: list) -> torch.Tensor:
        """The slices' partial sums through the compressed two-shot path."""
        return self.sum.run(torch.stack(parts)).clone()

    def forward(self, y: torch.Tensor, h: torch.Tensor, gate: torch.Tensor | None = None):
        """y, h bf16 [tokens, d] -> (out bf16 [tokens, d], h1).  ``gate``: this
        call's, in place of the block's."""
        gate = self.gate if gate is None else gate
        h1, codes, scale = api.rmsnorm_gate_residual_fp8(y, h, self.gain_post, self.gain_pre, gate,
                                                         self.residual_scale, self.eps)
        u = [api.fp8_gemm(codes, scale, w[0], w[1]) for w in self.up]
        out = self._reduce([api.fp8_linear(torch.nn.functional.silu(up), w[0], w[1]) for up, w in zip(u, self.down)])
        self._saved = (y, h, h1, u, gate)
        return out, h1

    def backward(self, dout: torch.Tensor, dh1: torch.Tensor):
        """Gradients at out and h1 -> (dy, dh, dgain_post, dgain_pre, dgate);
        the weights' gradients are added to the FP8 main gradients.  Each
        forward pass serves one backward pass: a second would add the same
        micro-batch's gradients again."""
        if self._saved is None:
            raise RuntimeError("backward() without a forward() of its own")
        (y, h, h1, us, gate), self._saved = self._saved, None
        _, n = api.rmsnorm_gate_residual(y, h, self.gain_post, self.gain_pre, gate, self.residual_scale, self.eps)
        dns = []
        for p, u in enumerate(us):
            s = torch.sigmoid(u.float())
            a = (u.float() * s).bfloat16()
            da, dw = api.fp8_linear_backward(dout, a, self.down[p][2], self.down[p][3], dw_dtype=torch.bfloat16)
            api.agoq_fp8_accumulate(*self.main_down[p], dw)
            du = (da.float() * s * (1.0 + u.float() * (1.0 - s))).bfloat16()
            dn, dw = api.fp8_linear_backward(du, n, self.up[p][2], self.up[p][3], dw_dtype=torch.bfloat16)
            api.agoq_fp8_accumulate(*self.main_up[p], dw)
            dns.append(dn)
        dn = self._reduce(dns)
        return api.rmsnorm_gate_residual_backward(dn, dh1, y, h1, self.gain_post, self.gain_pre, gate,
                                                  self.residual_scale, self.eps)
