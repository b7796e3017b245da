"""The norms around a block with every eps the calls accept, down to fp32's
subnormals, for rows whose mean square eps decides: rows of zeros, tiny rows,
and token counts that leave a CTA's pair of rows half empty.

The bounds are those of test_gpu_norms: fp32 arithmetic with sums of d (or T)
terms in any order, each addition off by at most 2^-23, and half a bf16 step.
1 / sqrt(eps) may be 2e22 here; a gradient that multiplies two of them would
leave fp32's range, so y and h_new are zero in different rows."""

import pytest
import torch

import fp8_reference as R
from fp8_communication_compression_gb300 import api
from test_gpu_norms import MODES, half_step, make

pytestmark = pytest.mark.gpu


def fp32(v):
    return float(torch.tensor(v, dtype=torch.float32))


@pytest.mark.parametrize("eps", [1e-20, 1e-27, 1e-33, 2e-38, 1e-42])
@pytest.mark.parametrize("T,d", [(1, 64), (3, 520), (5, 257), (9, 2560), (1, 4096), (161, 96), (3, 5120), (2, 8200),
                                 (3649, 2304)])
@pytest.mark.parametrize("mode", MODES)
def test_backward_with_a_small_eps(T, d, mode, eps):
    s = 0.7
    y, h2, gp, gq, gate = make(T, d, mode, 61)
    if T > 2:
        y[0] = 0                      # decided by eps alone
        h2[1] = 0
        y[2] *= 2.0 ** -40            # and the neighbourhood of eps
        h2[2] *= 2.0 ** -40
    g = torch.Generator().manual_seed(62)
    dn, dh2 = ((0.1 * torch.randn((T, d), generator=g)).bfloat16().cuda() for _ in range(2))
    if T > 2:
        dh2[2] = 0
    got = api.rmsnorm_gate_residual_backward(dn, dh2, y, h2, gp, gq, gate, s, eps)
    ref = R.norm_backward(dn, dh2, y, h2, gp, gq, gate, s, fp32(eps))
    mag = R.norm_backward(dn, dh2, y, h2, gp, gq, gate, s, fp32(eps), magnitude=True)
    u_row, u_sum = 4 * (d + 64) * 2.0 ** -23, (4 * (d + 64) + T) * 2.0 ** -23
    for name, a, b, m in zip(("dy", "dh", "dg_post", "dg_pre", "dgate"), got, ref, mag):
        if b is None:
            assert a is None
            continue
        tol = (u_sum if name in ("dg_post", "dg_pre") or mode == "channel" else u_row) * m
        if a.dtype == torch.bfloat16:
            tol = tol + half_step(b)
        assert torch.isfinite(a).all(), name
        assert ((a.cpu().double() - b).abs() <= tol).all(), name


@pytest.mark.parametrize("eps", [1e-27, 2e-38, 1e-42])
@pytest.mark.parametrize("T,d", [(1, 64), (3, 257), (5, 4096)])
def test_forward_with_a_small_eps(T, d, eps):
    y, h, gp, gq, gate = make(T, d, "token", 63)
    if T > 2:
        y[0] = 0
        y[1] = 0
        h[1] = 0
    h2, n = api.rmsnorm_gate_residual(y, h, gp, gq, gate, 0.7, eps)
    ref_h, ref_n = R.norm_forward(y, h, gp, gq, gate, 0.7, fp32(eps))
    u = (d + 64) * 2.0 ** -23
    mag = (0.7 * h.cpu().double()).abs() + (ref_h - 0.7 * h.cpu().double()).abs()
    assert ((h2.cpu().double() - ref_h).abs() <= half_step(ref_h) + u * mag).all()
    rn = (ref_n / torch.where(ref_h == 0, torch.ones_like(ref_h), ref_h)).abs()
    assert ((n.cpu().double() - ref_n).abs() <= half_step(ref_n) + u * (ref_n.abs() + rn * mag)).all()


def test_values_whose_squares_leave_the_range():
    # an infinite norm: the normalised values are zero, and the other rows are untouched
    T, d = 4, 320
    y, h, gp, gq, _ = make(T, d, "none", 64)
    ref_h, ref_n = api.rmsnorm_gate_residual(y, h, gp, gq, None, 0.5)
    y[1], h[2] = 1e20, -1e20
    h2, n = api.rmsnorm_gate_residual(y, h, gp, gq, None, 0.5)
    assert torch.equal(h2[1], (0.5 * h[1].float()).bfloat16())
    assert not n[2].any() and torch.isfinite(n).all()
    for r in (0, 3):
        assert torch.equal(h2[r], ref_h[r]) and torch.equal(n[r], ref_n[r])
