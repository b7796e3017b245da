"""Plain float64 forms of the block-scaled FP8 format, its products and the
norms around a block (torch on the CPU), for the tests."""

from __future__ import annotations

import math

import torch


def ceil_to(n: int, m: int) -> int:
    return -(-n // m) * m


def e4m3_round(v: torch.Tensor) -> torch.Tensor:
    """float64 values within +-448, rounded to the nearest E4M3 value, ties to
    the even code: steps of 2^(e - 3) in [2^e, 2^(e + 1)), 2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def block_exponent(amax: torch.Tensor) -> torch.Tensor:
    """Smallest E >= -127 with amax <= 448 2^E; 0 for amax = 0 (float64)."""
    E = torch.full(amax.shape, -127, dtype=torch.int64)
    while True:
        big = amax > torch.ldexp(torch.full_like(amax, 448.0), E)
        if not big.any():
            return torch.where(amax == 0, torch.zeros_like(E), E)
        E = E + big.long()


def code_values(codes: torch.Tensor) -> torch.Tensor:
    """uint8 E4M3 codes -> float64 values, from their bits."""
    c = codes.cpu().long()
    ex, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ex == 0, m * 2.0 ** -9, torch.ldexp(1.0 + m / 8.0, ex - 7))
    mag = torch.where((c & 127) == 127, torch.full_like(mag, math.nan), mag)
    return torch.where(c >= 128, -mag, mag)


def quantise(x: torch.Tensor, tiles: bool = False):
    """float64 [rows, cols] -> (values of the codes [rows, cols], exponents:
    [blocks, rows], or [blocks, row tiles] for 128 x 128 tiles)."""
    rows, cols = x.shape
    R, C = (ceil_to(rows, 128) if tiles else rows), ceil_to(cols, 128)
    p = torch.zeros((R, C), dtype=torch.float64)
    p[:rows, :cols] = x
    if tiles:
        E = block_exponent(p.view(R // 128, 128, C // 128, 128).abs().amax(dim=(1, 3)))
        full = E.repeat_interleave(128, 0).repeat_interleave(128, 1)
    else:
        E = block_exponent(p.view(rows, C // 128, 128).abs().amax(dim=2))
        full = E.repeat_interleave(128, 1)
    q = e4m3_round(torch.ldexp(p, -full))
    return q[:rows, :cols], E.t().contiguous()


def dequantised(x: torch.Tensor) -> torch.Tensor:
    """float64 [rows, cols] -> the values its quantised rows stand for."""
    q, E = quantise(x)
    return torch.ldexp(q, E.t().repeat_interleave(128, 1)[:, :q.shape[1]])


def scale_full(scale: torch.Tensor, rows: int, cols: int, tiles: bool) -> torch.Tensor:
    """Scale bytes [blocks, rows or row tiles] -> float64 [rows, cols]."""
    e = scale.cpu().long().t() - 127
    if tiles:
        e = e.repeat_interleave(128, 0)[:rows]
    s = torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e)
    s = torch.where(e == 128, torch.full_like(s, math.nan), s)
    return s.repeat_interleave(128, 1)[:, :cols]


def values(codes: torch.Tensor, scale: torch.Tensor, tiles: bool = False) -> torch.Tensor:
    """What codes [rows, P] and their scales stand for, float64."""
    rows, P = codes.shape
    return code_values(codes) * scale_full(scale, rows, P, tiles)


def gate_full(gate, T: int, d: int) -> torch.Tensor:
    return torch.ones((T, d), dtype=torch.float64) if gate is None else gate.cpu().double().expand(T, d)


def norm_forward(y, h, g_post, g_pre, gate, s: float, eps: float):
    y, h, g_post, g_pre = (t.cpu().double() for t in (y, h, g_post, g_pre))
    T, d = y.shape
    z = y / torch.sqrt((y * y).sum(1, keepdim=True) / d + eps) * g_post
    h2 = s * h + gate_full(gate, T, d) * z
    return h2, h2 / torch.sqrt((h2 * h2).sum(1, keepdim=True) / d + eps) * g_pre


def norm_backward(dn, dh2, y, h2, g_post, g_pre, gate, s: float, eps: float, magnitude: bool = False):
    """The gradients' formulas; with ``magnitude``, the sums of the absolute
    values of their terms (for error bounds)."""
    dn, dh2, y, h2, g_post, g_pre = (t.cpu().double() for t in (dn, dh2, y, h2, g_post, g_pre))
    T, d = y.shape
    w = gate_full(gate, T, d)
    ry = 1.0 / torch.sqrt((y * y).sum(1, keepdim=True) / d + eps)
    rh = 1.0 / torch.sqrt((h2 * h2).sum(1, keepdim=True) / d + eps)
    sign = -1.0
    if magnitude:
        dn, dh2, y, h2, g_post, g_pre, w = (t.abs() for t in (dn, dh2, y, h2, g_post, g_pre, w))
        s, sign = abs(s), 1.0
    u = dn * g_pre
    G = dh2 + rh * u + sign * h2 * rh ** 3 * (u * h2).sum(1, keepdim=True) / d
    v = G * w * g_post
    dy = ry * v + sign * y * ry ** 3 * (v * y).sum(1, keepdim=True) / d
    yg = y * ry * G
    dg_pre, dg_post = (dn * h2 * rh).sum(0), (yg * w).sum(0)
    dw = yg * g_post
    if gate is None:
        dgate = None
    elif gate.dim() == 1:
        dgate = dw.sum(0)
    elif gate.dtype == torch.float32:
        dgate = dw.sum(1, keepdim=True)
    else:
        dgate = dw
    return dy, s * G, dg_post, dg_pre, dgate
